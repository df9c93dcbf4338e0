"""Plain 64-bit forms of the serving operators, for the tests: numpy on the host, written
from the operators' definitions."""
import math

import numpy as np
import torch

import oracle

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0])
E4M3 = np.array([oracle.e4m3_value(c) for c in range(256)], np.float64)


def to_bf16(v):
    """float64/32 -> the float32 value of its nearest BF16 (v already float32-exact)."""
    bits = oracle.f32_to_bf16(np.ascontiguousarray(v, dtype=np.float32).reshape(-1))
    return (bits.astype(np.uint32) << 16).view(np.float32).reshape(np.shape(v))


def f32_of_bf16(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().float().numpy()


# ------------------------------------------------------------------ norm
def norm_reference(x, res, w, eps, options):
    """(z, y float32, codes, scales) of float32 arrays of BF16 values: the stated steps, the
    sum of squares exact."""
    z = to_bf16(x + res) if res is not None else x
    m, n = z.shape
    y = np.empty((m, n), np.float32)
    codes = np.empty((m, n), np.uint8)
    scales = np.empty((m, n // 128), np.float32)
    with np.errstate(all="ignore"):
        for i in range(m):
            row = z[i].astype(np.float64)
            total = math.fsum(row * row) if np.isfinite(row).all() else float(np.sum(row * row))
            r = np.float32(1.0 / np.sqrt(np.float64(total) / n + np.float64(np.float32(eps))))
            y[i] = (z[i] * r) * w
            for g in range(n // 128):
                part = np.ascontiguousarray(y[i, 128 * g:128 * g + 128])
                codes[i, 128 * g:128 * g + 128], scales[i, g] = fp8_block(part, options)
    return z, y, codes, scales


def fp8_block(part, options):
    import ctypes
    c = np.empty(part.size, np.uint8)
    s = oracle.lib().oracle_fp8_block(part.ctypes.data_as(ctypes.c_void_p), part.size, options,
                                      c.ctypes.data_as(ctypes.c_void_p))
    return c, np.float32(s)


# ------------------------------------------------------------------ rotary append
def rope_reference(x, positions, inv_freq, factor, interleaved):
    """BF16 values (float32) of the rotated heads: x [tokens][heads][d] float32."""
    half = inv_freq.size
    theta = positions.astype(np.float64)[:, None] * inv_freq
    c = (factor * np.cos(theta)).astype(np.float32)[:, None]
    s = (factor * np.sin(theta)).astype(np.float32)[:, None]
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    out = x.copy()
    with np.errstate(all="ignore"):
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., b] * c + x[..., a] * s
    rot = out[..., :2 * half]
    out[..., :2 * half] = to_bf16(rot) if rot.size else rot
    return out


def encode_rows(y, g):
    """NVFP4 of [tokens][heads][d] with a tensor scale per head: packed codes and scales."""
    t, h, d = y.shape
    codes = np.empty((t, h, d // 2), np.uint8)
    scales = np.empty((t, h, d // 16), np.uint8)
    for i in range(t):
        for j in range(h):
            for b in range(d // 16):
                sc, c = oracle.nvfp4_block(np.ascontiguousarray(y[i, j, 16 * b:16 * b + 16]), float(g[j]))
                c = np.asarray(c, np.uint8)
                codes[i, j, 8 * b:8 * b + 8] = c[0::2] | (c[1::2] << 4)
                scales[i, j, b] = sc
    return codes, scales


def decode_rows(codes, scales):
    """float64 E2M1 * E4M3 values (without the tensor scale)."""
    v = np.empty(codes.shape[:-1] + (codes.shape[-1] * 2,))
    v[..., 0::2], v[..., 1::2] = E2M1[codes & 15], E2M1[codes >> 4]
    with np.errstate(invalid="ignore"):
        return v * np.repeat(E4M3[scales], 16, axis=-1)


# ------------------------------------------------------------------ attention
def attention_reference(q, kc, ks, vc, vs, kg, vg, table, lens, starts, scale, window=0, sinks=0):
    """64-bit attention.  q [total][heads][d] float32; cache arrays [pages][kv][page][..]
    (host uint8); returns out, lse and how far each may be off (attention_bounds).  Rows of
    no sequence come back NaN."""
    total, hq, d = q.shape
    pages, hk, page = kc.shape[:3]
    out = np.full((total, hq, d), np.nan)
    mean_v, sum_v = np.zeros((total, hq, d)), np.zeros((total, hq, d))
    lse = np.full((total, hq), np.nan)
    big = np.zeros((total, hq))
    for b, n in enumerate(lens):
        lo, hi = int(starts[b]), int(starts[b + 1])
        if hi <= lo:
            continue
        n = int(n)
        at = np.array([table[b][t // page] for t in range(n)], np.int64)
        off = np.arange(n) % page
        pos = np.arange(n - (hi - lo), n)[:, None]
        key = np.arange(n)[None]
        see = key <= pos
        if window:
            see = see & ((key > pos - window) | (key < sinks))
        for h in range(hk):
            k = decode_rows(kc[at, h, off], ks[at, h, off]) * float(kg[h])
            v = decode_rows(vc[at, h, off], vs[at, h, off]) * float(vg[h])
            for j in range(h * (hq // hk), (h + 1) * (hq // hk)):
                qq = q[lo:hi, j].astype(np.float64)
                for i in range(hi - lo):
                    idx = np.nonzero(see[i])[0]
                    if idx.size == 0:
                        out[lo + i, j], lse[lo + i, j] = 0.0, -np.inf
                        continue
                    x = (k[idx] @ qq[i]) * scale
                    m = x.max()
                    p = np.exp(x - m)
                    out[lo + i, j] = p @ v[idx] / p.sum()
                    mean_v[lo + i, j] = p @ np.abs(v[idx]) / p.sum()
                    sum_v[lo + i, j] = np.abs(v[idx]).sum(0)
                    lse[lo + i, j] = m + np.log(p.sum())
                    big[lo + i, j] = (np.abs(k[idx]) @ np.abs(qq[i])).max() * scale
    return (out, lse, *attention_bounds(out, lse, mean_v, sum_v, big, d))


def attention_bounds(out, lse, mean_v, sum_v, big, d):
    """How far FP32 arithmetic with BF16 output may be off.  A score: its d products are
    exact and summed in FP32 (d roundings of at most 2^-24 of sum |q k|), then scaled, shifted
    and exponentiated (4 more roundings relative to a shifted score of at most twice the
    largest, and 2^-22 for the exponential): delta.  Weights are held in 11 significant bits
    (half a step 2^-12; 2^-11 counted) and their sum in FP32; numerator and denominator both
    carry delta.  Below FP16's normal range a weight is off by at most half its smallest
    subnormal, 2^-25, where the row's largest weight is at least 2^9 and so is the sum: 2^-34
    of sum |v| over the tokens seen.  All that is e; the output is then rounded to BF16: 2^-8
    of at most |out| + e (or half the smallest subnormal)."""
    delta = (d + 8) * 2.0 ** -24 * big[..., None] + 2.0 ** -22
    e = mean_v * (2 * delta + 2.0 ** -11) * 1.05 + 2.0 ** -34 * sum_v
    o = 2.0 ** -8 * (np.abs(out) + e) + e + 2.0 ** -60
    l = delta[..., 0] + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0.0))
    return o, l


def random_cache(rng, pages, hk, page, d, k_amp=1.0, v_amp=1.0):
    """Codes and scales of normal values (host arrays) and the heads' tensor scales."""
    out = []
    for amp in (k_amp, v_amp):
        g = (amp * (4.0 + rng.random(hk)) / 2688.0).astype(np.float32)
        z = rng.standard_normal((pages, hk, page, d // 16, 16)) * amp
        a = np.abs(z).max(-1)
        t = a / 6.0 / g[None, :, None, None].astype(np.float64)
        sc = oracle.e4m3_encode(np.minimum(t, 448.0).astype(np.float32).reshape(-1)).reshape(t.shape)
        step = E4M3[sc] * g[None, :, None, None]
        with np.errstate(all="ignore"):
            u = np.where(step[..., None] > 0, z / step[..., None], 0.0)
        c = oracle.e2m1_encode(u.astype(np.float32).reshape(-1)).reshape(pages, hk, page, d)
        out.append((np.ascontiguousarray(c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8), sc.astype(np.uint8), g))
    return out

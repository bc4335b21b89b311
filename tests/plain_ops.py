"""Plain numpy forms (64-bit unless a rule fixes fp32 steps) of the MX4 and cache operators, written from their
definitions in include/qmm.h, for the tests."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
ULP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}   # largest relative error of one rounding (bf16: 2^-9, doubled)


def mx4_quantize(x: np.ndarray):
    """fp32 [R, K] -> (codes uint8 [R, K], scales uint8 [R, K/32])."""
    R, K = x.shape
    b = x.astype(np.float64).reshape(R, K // 32, 32)
    top = np.abs(b).max(-1)
    bad = ~np.isfinite(b).all(-1)
    _, e = np.frexp(np.where(bad, 0.0, top))
    e = np.where(top > 0, np.clip(e - 1 - 2 + 127, 0, 254), 0)
    e = np.where(bad, 255, e)
    v = np.where(bad[..., None], 0.0, b) * np.ldexp(1.0, np.where(bad, 0, 127 - e))[..., None]
    # nearest of the eight magnitudes, ties to the even code
    dist = np.abs(np.abs(v)[..., None] - E2M1[:8])
    best = dist.min(-1, keepdims=True)
    tied = dist == best
    lo = tied.argmax(-1)
    two = tied.sum(-1) > 1
    code = np.where(two & (lo % 2 == 1), lo + 1, lo)
    code = np.where(np.signbit(v), code + 8, code)
    code = np.where(bad[..., None], 0, code)
    return code.reshape(R, K).astype(np.uint8), e.astype(np.uint8)


def mx4_values(codes, scales):
    R, K = codes.shape
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(int) - 127))
    return (E2M1[codes].reshape(R, K // 32, 32) * s[..., None]).reshape(R, K)


def mx4_pack_codes(codes):
    return (codes[:, 0::2] | codes[:, 1::2] << 4).astype(np.uint8)


def mx4_scale_index(R, K):
    """Byte offset of the scale of (row, block) in the scales buffer."""
    r, b = np.arange(R)[:, None], np.arange(K // 32)[None, :]
    return (r // 128 * -(-K // 128) + b // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + b % 4


def mx4_scales_bytes(R, K):
    return -(-R // 128) * -(-K // 128) * 512


def mx4_pack_scales(scales, K, fill=0):
    R = scales.shape[0]
    buf = np.full(mx4_scales_bytes(R, K), fill, np.uint8)
    # blocks past K hold 0 for every row that exists
    K4 = -(-K // 128) * 128
    buf[mx4_scale_index(R, K4)] = 0
    buf[mx4_scale_index(R, K)] = scales
    return buf


def code_bytes(type_, D):
    return D if type_ == "q8_0" else D // 2


def token_bytes(type_, D):
    return code_bytes(type_, D) + D // 32 * 2


def block_quantize(type_, x: np.ndarray):
    """fp32 [..., D] -> (code bytes uint8 [..., code_bytes], scales fp16 [..., D/32]) with the fp32 steps of the rules."""
    f = np.float32
    b = x.astype(f).reshape(*x.shape[:-1], -1, 32)
    bad = ~np.isfinite(b).all(-1)
    z = np.where(bad[..., None], f(0), b)
    a = np.abs(z)
    top = a.max(-1)
    with np.errstate(all="ignore"):
        if type_ == "q8_0":
            d = (top * (f(1) / f(127))).astype(f)
        else:
            m = np.take_along_axis(z, a.argmax(-1)[..., None], -1)[..., 0]     # the first on ties
            d = (m / f(-8)).astype(f)
        half = d.astype(np.float16)
        bad |= ~np.isfinite(half)
        inv = np.where(d != 0, f(1) / d, f(0)).astype(f)
        v = (z * inv[..., None]).astype(f)
        if type_ == "q8_0":
            v = np.where(np.isnan(v), f(0), v).astype(np.float64)
            q = np.clip(np.sign(v) * np.floor(np.abs(v) + 0.5), -127, 127)
            q = np.where(bad[..., None], 0, q).astype(np.int8)
            codes = q.view(np.uint8).reshape(*x.shape)
        else:
            v = (v + f(8.5)).astype(f)
            q = np.where(v >= 0, np.trunc(np.minimum(v, 15)), 0)
            q = np.where(bad[..., None], 0, np.where(np.isnan(q), 0, q)).astype(np.uint8)
            codes = (q[..., :16] | q[..., 16:] << 4).reshape(*x.shape[:-1], -1)
    return codes, np.where(bad, np.float16(np.nan), half)


def block_values(type_, codes, scales):
    """(code bytes, fp16 scales) -> fp64 values [..., D]."""
    n = scales.shape[-1]
    if type_ == "q8_0":
        q = codes.view(np.int8).reshape(*codes.shape[:-1], n, 32).astype(np.float64)
    else:
        c = codes.reshape(*codes.shape[:-1], n, 16)
        q = np.concatenate((c & 15, c >> 4), -1).astype(np.float64) - 8
    return (q * scales.astype(np.float64)[..., None]).reshape(*codes.shape[:-1], 32 * n)


def cache_views(cache: np.ndarray, type_, H, D, P):
    """uint8 [n_pages, H, chunk] -> views of the codes [n_pages, H, P, bytes] and fp16 scales [n_pages, H, P, D/32]."""
    n = P * code_bytes(type_, D)
    pages = cache.shape[0]
    codes = cache[..., :n].reshape(pages, H, P, -1)
    scales = cache[..., n:].copy().view(np.float16).reshape(pages, H, P, -1)
    return codes, scales


def make_chunks(type_, codes, scales):
    """codes [pages, H, P, bytes], scales [pages, H, P, D/32] -> cache bytes [pages, H, chunk]."""
    pages, H = codes.shape[:2]
    s = np.ascontiguousarray(scales.astype(np.float16)).view(np.uint8)
    return np.concatenate((codes.reshape(pages, H, -1), s.reshape(pages, H, -1)), -1)


def attend(q, k, v, seen, scale):
    """fp64: q [rows, D], k, v [n, D], seen bool [rows, n] -> (out, sum p|v|, lse, largest scale*sum|q||k| over the seen)."""
    out = np.zeros((q.shape[0], v.shape[1]))
    mag = np.zeros_like(out)
    lse = np.full(q.shape[0], -np.inf)
    big = np.zeros(q.shape[0])
    for i in range(q.shape[0]):
        at = np.nonzero(seen[i])[0]
        if at.size == 0:
            continue
        s = scale * (k[at] @ q[i])
        top = s.max()
        with np.errstate(invalid="ignore"):
            p = np.exp(s - top)
            out[i] = p @ v[at] / p.sum()
            mag[i] = p @ np.abs(v[at]) / p.sum()
            lse[i] = top + np.log(p.sum())
            big[i] = abs(scale) * (np.abs(k[at]) @ np.abs(q[i])).max()
    return out, mag, lse, big

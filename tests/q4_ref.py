"""Plain 64-bit implementation of the 4-bit cache's format and of windowed
attention, for the tests: numpy, written from the format's definition in
include/pa.h, sharing nothing with the kernels."""
import numpy as np
import torch


def f32(x):
    """Round to fp32 and widen back."""
    return np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


def bf16_toward(x, up):
    """The nearest bf16 at or above (up) / at or below x, for fp32-representable x."""
    b = np.asarray(x, np.float64).astype(np.float32).view(np.uint32).astype(np.int64)
    low = b & 0xffff
    neg = (b >> 31) != 0
    away = (low != 0) & (neg != up)          # the larger magnitude is the one asked for
    b = (b & 0xffff0000) + np.where(away, 0x10000, 0)
    return b.astype(np.uint32).view(np.float32).astype(np.float64)


def quantise(x, group):
    """codes [..., hd] (ints), steps and minima [..., groups] of fp32 rows (float64 array)."""
    x = np.asarray(x, np.float64)
    g = x.reshape(*x.shape[:-1], -1, group)
    with np.errstate(all="ignore"):
        bad = ~(np.abs(g) < 2.0 ** 126).all(-1)
        g = np.where(bad[..., None], 0.0, g)
        m = bf16_toward(g.min(-1), False)
        far = f32(g.max(-1) - m)
        s = np.maximum(bf16_toward(f32(far / 15), True), 2.0 ** -126)
        s = np.where(far > 0, s, 0.0)
        inv = np.where(s > 0, f32(1 / np.where(s > 0, s, 1.0)), 0.0)
        codes = np.rint(f32(f32(g - m[..., None]) * inv[..., None])).astype(np.int64)
    assert codes.min(initial=0) >= 0 and codes.max(initial=0) <= 15
    return codes.reshape(x.shape), np.where(bad, 0.0, s), np.where(bad, np.nan, m)


def spot(hd):
    """(byte, shift) of each value of a row's codes."""
    d = np.arange(hd)
    u, j = d // 4, d % 4
    w, h, g = u // 16, u // 8 % 2, u % 8
    return (g * (hd // 64) + w) * 4 + h * 2 + j // 2, j % 2 * 4


def page_bytes(hd, bs, group):
    return bs * (hd // 2 + 4 * (hd // group))


def bf16_bits(x):
    b = torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)
    return b.view(torch.int16).numpy().astype(np.uint16)


def write(cache, x, slots, bs, group):
    """Write rows x [T, H, hd] (float64) into cache uint8 [nb, H, page_bytes] (numpy, in place)."""
    hd = x.shape[-1]
    codes, s, m = quantise(x, group)
    byte, shift = spot(hd)
    cut = bs * hd // 2
    for t, slot in enumerate(slots):
        if slot < 0 or slot >= cache.shape[0] * bs:
            continue
        b, r = divmod(int(slot), bs)
        for h in range(x.shape[1]):
            row = np.zeros(hd // 2, np.uint8)
            np.bitwise_or.at(row, byte, (codes[t, h] << shift).astype(np.uint8))
            cache[b, h, r * (hd // 2):(r + 1) * (hd // 2)] = row
            par = np.stack([bf16_bits(s[t, h]), bf16_bits(m[t, h])], -1).reshape(-1)
            n = par.size * 2
            cache[b, h, cut + r * n:cut + (r + 1) * n] = par.view(np.uint8)


def values(cache, bs, hd, group):
    """fp64 [nb, H, bs, hd] of everything a cache holds."""
    cache = np.ascontiguousarray(cache)
    nb, H = cache.shape[:2]
    cut = bs * hd // 2
    raw = cache[..., :cut].reshape(nb, H, bs, hd // 2)
    byte, shift = spot(hd)
    codes = (raw[..., byte] >> shift) & 15
    par = torch.from_numpy(np.ascontiguousarray(cache[..., cut:])).view(torch.bfloat16).double().numpy()
    par = np.repeat(par.reshape(nb, H, bs, hd // group, 2), group, axis=3)
    return codes * par[..., 0] + par[..., 1]


def attend(q, kv, vv, tables, lens, scale, bs, window=0, sinks=0):
    """fp64 attention [S, Hq, hd]: q [S, Hq, hd]; kv, vv [nb, H, bs, hd] float64."""
    S, Hq, hd = q.shape
    H = kv.shape[1]
    out = np.zeros((S, Hq, hd))
    for i in range(S):
        n = int(lens[i])
        t = np.arange(n)
        if window:
            t = t[(t >= n - window) | (t < sinks)]
        if not len(t):
            continue
        blk = tables[i][t // bs]
        ok = (blk >= 0) & (blk < kv.shape[0])      # a bad block id reads as zeros
        k = np.where(ok[:, None, None], kv[np.where(ok, blk, 0), :, t % bs], 0.0)
        v = np.where(ok[:, None, None], vv[np.where(ok, blk, 0), :, t % bs], 0.0)
        for h in range(Hq):
            kh = h // (Hq // H)
            x = scale * (k[:, kh] @ q[i, h])
            p = np.exp(x - x.max())
            out[i, h] = (p @ v[:, kh]) / p.sum()
    return out

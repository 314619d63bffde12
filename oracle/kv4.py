"""The 4-bit key/value cache in fp64 (test infrastructure only): quantisation, decode, eviction.

"Lecture 8 · GPU Performance & FlashAttention" §8.1 quantises blocks with a scale each and §8.2
decodes over a cache; the pages fix no 4-bit format.  The format used here holds, for every 64
channels of a row, a step and a middle in fp16 and a 4-bit code c per channel that stands for
middle + step (c - 8).  The decisions that produce codes are taken in fp32 (the precision of the
quantising kernel), so that codes compare bit for bit; everything else is fp64.
"""

from __future__ import annotations

import numpy as np

__all__ = ["GROUP", "LIMIT", "quantize_rows", "dequantize_rows", "pack_blocks", "unpack_blocks", "decode64", "evict"]

GROUP = 64
LIMIT = 32768.0


def _fp16_up(x):
    """fp16 >= the fp32 x, the nearest such."""
    with np.errstate(over="ignore"):
        h = x.astype(np.float16)
    return np.where(h.astype(np.float32) < x, np.nextafter(h, np.float16(np.inf)), h).astype(np.float16)


def quantize_rows(x):
    """x [..., d] fp32 -> codes [..., d] uint8, step and middle [..., d / 64] fp16."""
    x = np.asarray(x, np.float32)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    bad = ~np.all(np.abs(g) <= LIMIT, axis=-1)
    g = np.where(bad[..., None], np.float32(0), g)
    lo, hi = g.min(-1), g.max(-1)
    step = _fp16_up(((hi - lo).astype(np.float32) / np.float32(15)).astype(np.float32))
    s = step.astype(np.float32)
    middle = (lo + np.float32(8) * s).astype(np.float32).astype(np.float16)
    m = middle.astype(np.float32)
    safe = np.where(s > 0, s, np.float32(1))
    t = ((g - m[..., None]).astype(np.float32) / safe[..., None]).astype(np.float32)
    codes = np.clip(np.rint(t), -8, 7) + 8
    codes = np.where((s > 0)[..., None], codes, 8).astype(np.uint8)
    nan = np.float16(np.nan)
    return (np.where(bad[..., None], 8, codes).astype(np.uint8).reshape(x.shape), np.where(bad, nan, step),
            np.where(bad, nan, middle))


def dequantize_rows(codes, step, middle):
    """The fp64 values that the codes stand for."""
    c = np.asarray(codes, np.float64).reshape(*codes.shape[:-1], -1, GROUP) - 8
    return (np.asarray(middle, np.float64)[..., None] + np.asarray(step, np.float64)[..., None] * c).reshape(codes.shape)


def pack_blocks(k, v):
    """(codes, step, middle) of K and of V, [..., C, d] with C a multiple of 64 -> bytes [..., C / 64, 72 d]."""
    parts = {}
    for name, (codes, step, middle) in (("k", k), ("v", v)):
        lead, C = codes.shape[:-2], codes.shape[-2]
        by = (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)
        par = np.stack((step, middle), -1).astype(np.float16).view(np.uint8)
        parts[name] = by.reshape(*lead, C // 64, -1), par.reshape(*lead, C // 64, -1)
    return np.concatenate((parts["k"][0], parts["v"][0], parts["k"][1], parts["v"][1]), -1)


def unpack_blocks(blocks):
    """The inverse: bytes [..., nb, 72 d] -> ((codes, step, middle) of K, the same of V)."""
    d, lead, nb = blocks.shape[-1] // 72, blocks.shape[:-2], blocks.shape[-2]
    out = []
    for code_at, par_at in ((0, 64 * d), (32 * d, 68 * d)):
        by = blocks[..., code_at:code_at + 32 * d].reshape(*lead, nb * 64, d // 2)
        codes = np.empty((*lead, nb * 64, d), np.uint8)
        codes[..., 0::2], codes[..., 1::2] = by & 15, by >> 4
        par = np.ascontiguousarray(blocks[..., par_at:par_at + 4 * d]).view(np.float16).reshape(*lead, nb * 64, d // 64, 2)
        out.append((codes, par[..., 0], par[..., 1]))
    return out


def decode64(q, k, v, lens, scale, causal):
    """O, L and the probability sums [B, Hkv, C] of q [B, H, Nq, d] over k, v [B, Hkv, C, d]; sequence b has
    lens[b] slots, causal row i sees the first lens[b] - Nq + i + 1.  Also the largest |q| . |k| a row
    meets (times scale), which bounds the rounding of its scores."""
    B, H, Nq, d = q.shape
    hkv, C = k.shape[1], k.shape[2]
    o, L = np.zeros(q.shape), np.full((B, H, Nq), -np.inf)
    w, mag = np.zeros((B, hkv, C)), np.zeros((B, H, Nq))
    for b in range(B):
        for h in range(H):
            for i in range(Nq):
                n = int(lens[b]) - Nq + i + 1 if causal else int(lens[b])
                if n <= 0:
                    continue
                kk, vv = k[b, h * hkv // H, :n], v[b, h * hkv // H, :n]
                s = scale * (kk @ q[b, h, i])
                mag[b, h, i] = scale * (np.abs(kk) @ np.abs(q[b, h, i])).max()
                m = s.max()
                p = np.exp(s - m)
                L[b, h, i] = m + np.log(p.sum())
                p /= p.sum()
                o[b, h, i] = p @ vv
                w[b, h * hkv // H, :n] += p
    return o, L, w, mag


def evict(weights, n, keep, recent):
    """Slots of one head that stay: the newest `recent` of n and the heaviest others (ties: the lowest
    slot; NaN counts as the largest), ascending."""
    if n <= keep:
        return np.arange(n)
    old = n - recent
    w = np.asarray(weights[:old], np.float64)
    rank = sorted(range(old), key=lambda j: (0.0 if np.isnan(w[j]) else 1.0, 0.0 if np.isnan(w[j]) else -w[j], j))
    return np.array(sorted(rank[:keep - recent]) + list(range(old, n)), dtype=np.int64)

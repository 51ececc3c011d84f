"""Writing tokens into an INT4 KV cache, reading rows back, and attention of a
batch over a shared prefix and each sequence's own tokens (test infrastructure).

The cache is kept here as plain rows: codes uint8 [B, Hkv, cap, D] and scales
and zeros fp16 [B, Hkv, cap], one INT4 asymmetric group per row with the
quantizer of the weights (oracle/formats.py). `key_words` and `value_words`
give the packed layouts: K codes a token a row (element d in nibble d % 8 of
word d / 8), V codes in blocks of 8 tokens (token t in nibble t % 8). All
arithmetic beyond the quantizer's own fp32 steps is fp64.
"""

import numpy as np

from . import formats


def append(cache, rows, starts, offsets):
    """Write packed rows fp32 [T, Hkv, D] into one cache (codes, scales,
    zeros), in place; positions outside the capacity are dropped."""
    codes, scales, zeros = cache
    cap, d = codes.shape[2], codes.shape[3]
    for b, first in enumerate(starts):
        for i, t in enumerate(range(offsets[b], offsets[b + 1])):
            pos = first + i
            if 0 <= pos < cap:
                q, s, z = formats.int4_quantize(np.asarray(rows[t], np.float32), d)
                codes[b, :, pos] = q
                scales[b, :, pos] = s[:, 0]
                zeros[b, :, pos] = z[:, 0]


def read(cache, starts, offsets, total):
    """Exact fp64 rows [total, Hkv, D] (zeros outside the capacity)."""
    codes, scales, zeros = cache
    cap = codes.shape[2]
    out = np.zeros((total,) + (codes.shape[1], codes.shape[3]))
    for b, first in enumerate(starts):
        for i, t in enumerate(range(offsets[b], offsets[b + 1])):
            pos = first + i
            if 0 <= pos < cap:
                out[t] = (codes[b, :, pos].astype(np.float64)
                          - zeros[b, :, pos].astype(np.float64)[:, None]) * \
                    scales[b, :, pos].astype(np.float64)[:, None]
    return out


def key_words(codes):
    """uint8 [B, Hkv, cap, D] -> uint32 [B, Hkv, cap, D / 8]."""
    b, h, n, d = codes.shape
    return formats.int4_pack(codes.reshape(-1, d)).reshape(b, h, n, d // 8)


def value_words(codes):
    """uint8 [B, Hkv, cap, D] -> uint32 [B, Hkv, ceil(cap / 8), D]."""
    b, h, n, d = codes.shape
    full = np.zeros((b, h, (n + 7) // 8 * 8, d), np.uint32)
    full[:, :, :n] = codes
    out = np.zeros((b, h, (n + 7) // 8, d), np.uint32)
    for t in range(8):
        out |= full[:, :, t::8] << np.uint32(4 * t)
    return out


def prefix_attention(q, prefix_k, prefix_v, k_cache, v_cache, lengths, prefix_len):
    """fp64 attention of q [B, Hq, D] over the first prefix_len rows of the
    prefix caches (codes [1, Hkv, P, D], ...) and each sequence's own first
    lengths[b] rows; zeros where a sequence has no row at all."""
    def rows(cache, b, h, n):
        c, s, z = cache
        return (c[b, h, :n].astype(np.float64) - z[b, h, :n].astype(np.float64)[:, None]) * \
            s[b, h, :n].astype(np.float64)[:, None]
    q = np.asarray(q, np.float64)
    b_, hq, d = q.shape
    hkv = k_cache[0].shape[1]
    r = hq // hkv
    out = np.zeros_like(q)
    for h in range(hkv):
        kp, vp = rows(prefix_k, 0, h, prefix_len), rows(prefix_v, 0, h, prefix_len)
        for b in range(b_):
            k = np.concatenate([kp, rows(k_cache, b, h, lengths[b])])
            v = np.concatenate([vp, rows(v_cache, b, h, lengths[b])])
            if len(k) == 0:
                continue
            s = q[b, h * r:(h + 1) * r] @ k.T / np.sqrt(d)
            e = np.exp(s - s.max(axis=1, keepdims=True))
            out[b, h * r:(h + 1) * r] = (e @ v) / e.sum(axis=1, keepdims=True)
    return out

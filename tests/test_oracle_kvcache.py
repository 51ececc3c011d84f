"""Pins of the cache oracle: the packed layouts, append against the row quantizer,
read-back error, and attention against a plain softmax over concatenated rows."""

import numpy as np
import torch

from oracle import formats, kvcache

D = 128


def _cache(b, h, cap):
    return (np.zeros((b, h, cap, D), np.uint8), np.ones((b, h, cap), np.float16),
            np.zeros((b, h, cap), np.float16))


def test_layouts_place_every_code():
    codes = np.random.RandomState(0).randint(0, 16, (2, 3, 13, D)).astype(np.uint8)
    k, v = kvcache.key_words(codes), kvcache.value_words(codes)
    assert k.shape == (2, 3, 13, D // 8) and v.shape == (2, 3, 2, D)
    for t, d in ((0, 0), (7, 127), (8, 5), (12, 64)):
        assert np.array_equal((k[:, :, t, d // 8] >> np.uint32(4 * (d % 8))) & 15, codes[:, :, t, d])
        assert np.array_equal((v[:, :, t // 8, d] >> np.uint32(4 * (t % 8))) & 15, codes[:, :, t, d])
    assert not (v[:, :, 1] >> np.uint32(20)).any()  # tokens 13 .. 15 do not exist


def test_append_and_read_ragged():
    r = np.random.RandomState(1)
    cache = _cache(3, 2, 9)
    before = [a.copy() for a in cache]
    rows = r.randn(8, 2, D).astype(np.float32)
    starts, offsets = [0, 7, 4], [0, 3, 3, 8]       # 3 tokens, none, 5 of which 5 fit
    kvcache.append(cache, rows, starts, offsets)
    q, s, z = formats.int4_quantize(rows[4], D)
    assert np.array_equal(cache[0][2, :, 5], q) and np.array_equal(cache[1][2, :, 5], s[:, 0])
    for a, old in zip(cache, before):
        assert np.array_equal(a[1], old[1]) and np.array_equal(a[0, :, 3:], old[0, :, 3:])
    back = kvcache.read(cache, starts, offsets, 8)
    step = (np.maximum(rows.max(-1), 0) - np.minimum(rows.min(-1), 0)) / 15
    # half a step of the code and of the zero point, and the scale's rounding on 15 codes
    assert (np.abs(back - rows) <= step[..., None] * (1 + 15 * 2.0 ** -11)).all()


def test_positions_outside_the_cache():
    cache = _cache(1, 1, 4)
    rows = np.random.RandomState(2).randn(6, 1, D).astype(np.float32)
    kvcache.append(cache, rows, [-1], [0, 6])       # positions -1 .. 4: four of them exist
    back = kvcache.read(cache, [-1], [0, 6], 6)
    assert not back[0].any() and not back[5].any() and back[1:5].any(axis=(1, 2)).all()


def test_attention_is_softmax_over_both_caches():
    r = np.random.RandomState(3)
    b, hq, hkv, p, cap = 3, 4, 2, 6, 5
    caches = []
    for n, tokens in ((1, p), (1, p), (b, cap), (b, cap)):
        c = _cache(n, hkv, tokens)
        rows = r.randn(n * tokens, hkv, D).astype(np.float32)
        kvcache.append(c, rows, [0] * n, list(range(0, n * tokens + 1, tokens)))
        caches.append((c, kvcache.read(c, [0] * n, list(range(0, n * tokens + 1, tokens)),
                                       n * tokens).reshape(n, tokens, hkv, D)))
    (pk, pkr), (pv, pvr), (k, kr), (v, vr) = caches
    q = r.randn(b, hq, D)
    lengths = [0, 2, 5]
    out = kvcache.prefix_attention(q, pk, pv, k, v, lengths, p - 1)
    for i, n in enumerate(lengths):
        for h in range(hq):
            kk = np.concatenate([pkr[0, :p - 1, h // 2], kr[i, :n, h // 2]])
            vv = np.concatenate([pvr[0, :p - 1, h // 2], vr[i, :n, h // 2]])
            w = torch.softmax(torch.from_numpy(kk @ q[i, h]) / D ** 0.5, 0).numpy()
            assert np.allclose(out[i, h], w @ vv, rtol=1e-12, atol=1e-12)
    assert not kvcache.prefix_attention(q, pk, pv, k, v, [0] * b, 0).any()

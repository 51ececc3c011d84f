"""How exact the shared-prefix attention is, by kernel and type.

The prefix on mma.sync, own tokens, and the prefix on tcgen05 for fp16 queries multiply
exact operands: a score is off by the fp32 sums only (tcgen05: by 2^-15 of itself too, a
scale's low bits are rounded to bf16) and a value by nothing (2^-15). What is left is each
weight's rounding to fp16 and the output's own. tcgen05 with bf16 queries rounds K and V
to fp16 as well.

Element bound, with p the exact weights, s the scores, A = sum p |v|, sv the values' scales:
  2^-11 A             weights in fp16's normal range
  2^-23 n 15 max(p sv)   smaller ones: 2^-25 of a weight whose largest is at least 2^-1/2,
                      twice where a tile's bound moved after they were rounded
  sum p |v| (e^d - 1) and the same of the denominator, d = 2^-17 mag + 2^-21 max(|s|, 24)
                      (fp32 sums of 128 products, mag = sum |q k| / sqrt(D); the exponent),
                      and on tcgen05 2^-15 |s| and 2^-15 A (exact operands), or
                      2^-11 mag and 2^-11 A (rounded ones)
  2^-20 A             the exponentials and the fp32 sums of the products
then the output's half step.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

D = 128
BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def wq():
    from bit_weight_quantized_weights_b200 import binding
    return binding


@pytest.fixture
def on(wq):
    yield wq.wq_test_set_prefix_path
    wq.wq_test_set_prefix_path(0)


def _rows(part, is_value):
    """fp64 rows [B, H, n, D] and scales of a cache."""
    w, s, z = (t.cpu().numpy() for t in part)
    w = w.view(np.uint32)
    c = np.stack([(w >> np.uint32(4 * i)) & 15 for i in range(8)], 3 if is_value else -1)
    n = s.shape[2]
    c = c.reshape(s.shape[0], s.shape[1], -1, D)[:, :, :n].astype(np.float64)
    return (c - z.astype(np.float64)[..., None]) * s.astype(np.float64)[..., None], \
        s.astype(np.float64)


def _attend(q, k, v):
    """q [.., R, D], k and v [n, D] -> (scores, weights, outputs), fp64."""
    s = q @ k.T / np.sqrt(D)
    p = np.exp(s - s.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    return s, p, p @ v


def _bound(q, k, v, sv, tcgen05, exact, dtype):
    s, p, want = _attend(q, k, v)
    mag = np.abs(q) @ np.abs(k).T / np.sqrt(D)
    d = 2.0 ** -17 * mag + 2.0 ** -21 * np.maximum(np.abs(s), 24.0)
    rel = 2.0 ** -11 + 2.0 ** -20
    if tcgen05:
        d += 2.0 ** -15 * np.abs(s) if exact else 2.0 ** -11 * mag
        rel += 2.0 ** -15 if exact else 2.0 ** -11
    moved = p * np.expm1(d)
    slack = rel * (p @ np.abs(v)) + 2.0 ** -23 * len(k) * 15 * (p * sv).max(-1, keepdims=True) + \
        moved @ np.abs(v) + np.abs(want) * moved.sum(-1, keepdims=True)
    half = torch.finfo(dtype).eps / 2
    return want, slack + half * (np.abs(want) + slack) + (2.0 ** -25 if dtype == FP16 else 1e-30)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("path", [1, 2])
@pytest.mark.parametrize("rows", [8, 40])                # 64 and 320 rows: one, two row tiles
@pytest.mark.parametrize("ratio", [1.7, 2.0, 2.3, 2.6, 2.9])
def test_a_bound_that_moves_within_a_tile(wq, on, path, rows, ratio, dtype):
    """32 keys of score 0, 64 of scores 6 to 9 (base 2) whose values are 1, then one key far
    above them whose value is 0: the output is the 64 keys' share, whose weights were
    rounded against the bound of the first keys before the last one moved it."""
    on(path)
    n, hq = 128, 8
    k = torch.zeros(1, 1, n, D)
    v = torch.zeros(1, 1, n, D)
    base = 1.0 / (1.4426950408889634 * np.sqrt(D))       # of q = 1: one step of the exponent
    k[0, 0, 32:96] = 8.0 * base
    v[0, 0, 32:96] = 1.0
    k[0, 0, 100] = 8.0 * base * ratio
    # q's rows scale the scores: 6 to 9 for the 64 keys (10 with the values' scales)
    q = torch.linspace(0.8, 1.2, rows * hq)[:, None].expand(-1, D).reshape(rows, hq, D)
    q = q.to(dtype).cuda()
    pre = wq.kv_quantize_keys(k.cuda()), wq.kv_quantize_values(v.cuda())
    own = wq.kv_cache_alloc(rows, 1, 1)
    none = torch.zeros(rows, dtype=torch.int32, device="cuda")
    got = wq.wq_prefix_attention(q, *pre, *own, none).double().cpu().numpy()
    (kk, _), (vv, sv) = _rows(pre[0], False), _rows(pre[1], True)
    want, bound = _bound(q.double().cpu().numpy(), kk[0, 0], vv[0, 0], sv[0, 0], path == 2,
                         dtype == FP16, dtype)
    over = np.abs(got - want) / bound
    worst = float(over.max())
    assert worst <= 1, "%d of %d off, worst %.2f of the bound" % ((over > 1).sum(), over.size,
                                                                  worst)


@pytest.mark.parametrize("where,path,dtype,spread", [
    ("prefix", 1, FP16, 4.0), ("prefix", 1, BF16, 12.0), ("prefix", 2, FP16, 4.0),
    ("own", 1, FP16, 4.0), ("own", 1, BF16, 12.0)])
def test_operands_are_exact(wq, on, where, path, dtype, spread):
    """Scores of a standard deviation `spread`: rounding K and V to fp16 once would move the
    weights by more than their own rounding and the output's together. Element by element,
    and as a whole: a weight's rounding is off by at most 2^-10 / sqrt(12) of it (rms, worst
    mantissa), independent of the others; the output's by step / sqrt(12). 5% on top for the
    sample: 16384 outputs for the one, 128 rows of a few weights for the other, which is
    counted at its worst mantissa (1.4 times its mean)."""
    on(path)
    b, hq, hkv, n = 8, 16, 2, 1500
    g = torch.Generator().manual_seed(77)
    parts = 1 if where == "prefix" else b
    k = torch.randn(parts, hkv, n, D, generator=g) * spread
    v = torch.randn(parts, hkv, n, D, generator=g)
    q = torch.randn(b, hq, D, generator=g).to(dtype).cuda()
    cache = wq.kv_quantize_keys(k.cuda()), wq.kv_quantize_values(v.cuda())
    if where == "prefix":
        none = torch.zeros(b, dtype=torch.int32, device="cuda")
        got = wq.wq_prefix_attention(q, *cache, *wq.kv_cache_alloc(b, hkv, 1), none)
    else:
        got = wq.wq_prefix_attention(q, None, None, *cache,
                                     torch.full((b,), n, dtype=torch.int32, device="cuda"))
    got = got.double().cpu().numpy().reshape(b, hkv, hq // hkv, D)
    qn = q.double().cpu().numpy().reshape(b, hkv, hq // hkv, D)
    (kk, _), (vv, sv) = _rows(cache[0], False), _rows(cache[1], True)
    error = limit = rounded = 0.0
    for i in range(b):
        for h in range(hkv):
            j = i % parts
            want, bound = _bound(qn[i, h], kk[j, h], vv[j, h], sv[j, h], path == 2, True, dtype)
            assert (np.abs(got[i, h] - want) <= bound).all(), (i, h)
            _, p, _ = _attend(qn[i, h], kk[j, h], vv[j, h])
            step = torch.finfo(dtype).eps * 2.0 ** np.floor(np.log2(np.abs(want)))
            error += ((got[i, h] - want) ** 2).sum()
            limit += (step ** 2 / 12).sum() + 2.0 ** -20 / 12 * (p ** 2 @ vv[j, h] ** 2).sum()
            half = [t.astype(np.float16).astype(np.float64) for t in (kk[j, h], vv[j, h])]
            rounded += ((_attend(qn[i, h], *half)[2] - want) ** 2).sum() + (step ** 2 / 12).sum()
    assert error <= 1.05 ** 2 * limit, (error / limit) ** 0.5
    # the bound tells: the oracle with rounded operands (and exact weights) is beyond it
    assert rounded > 1.05 ** 2 * limit, (rounded / limit) ** 0.5


@pytest.mark.parametrize("where,path", [("prefix", 1), ("prefix", 2), ("own", 1)])
def test_many_keys_far_below_one_keep_their_precision(wq, on, where, path):
    """One key (the first) about 2^18 above 20000 others, of value 0, as a key that only
    collects weight: the output is the others' 7%, and their weights, 2^-18 of the largest,
    are rounded as finely as any (the bound of test_operands_are_exact)."""
    on(path)
    b, hq, hkv, n = 2, 8, 1, 20000
    g = torch.Generator().manual_seed(78)
    parts = 1 if where == "prefix" else b
    k = torch.randn(parts, hkv, n, D, generator=g) * 0.1
    v = torch.randn(parts, hkv, n, D, generator=g)
    k[:, :, 0] = 18.0 / (1.4426950408889634 * np.sqrt(D))    # of q = 1: 18 steps of the exponent
    v[:, :, 0] = 0.0
    q = (1.0 + 0.05 * torch.randn(b, hq, D, generator=g)).half().cuda()
    cache = wq.kv_quantize_keys(k.cuda()), wq.kv_quantize_values(v.cuda())
    if where == "prefix":
        none = torch.zeros(b, dtype=torch.int32, device="cuda")
        got = wq.wq_prefix_attention(q, *cache, *wq.kv_cache_alloc(b, hkv, 1), none)
    else:
        got = wq.wq_prefix_attention(q, None, None, *cache,
                                     torch.full((b,), n, dtype=torch.int32, device="cuda"))
    got, qn = got.double().cpu().numpy(), q.double().cpu().numpy()
    kk, vv = _rows(cache[0], False)[0], _rows(cache[1], True)[0]
    error = limit = 0.0
    for i in range(b):
        _, p, want = _attend(qn[i], kk[i % parts, 0], vv[i % parts, 0])
        assert p[:, 0].min() > 0.8
        step = 2.0 ** np.maximum(np.floor(np.log2(np.abs(want))) - 10, -24)
        error += ((got[i] - want) ** 2).sum()
        limit += (step ** 2 / 12).sum() + 2.0 ** -20 / 12 * (p ** 2 @ vv[i % parts, 0] ** 2).sum()
    assert error <= 1.05 ** 2 * limit, (error / limit) ** 0.5


def test_many_own_keys_far_below_one_in_a_full_batch(wq):
    """The same where every sequence and head has one range of keys: 2000 keys a head."""
    b, hq, hkv, n = 160, 8, 8, 2000
    g = torch.Generator().manual_seed(79)
    k = torch.randn(1, hkv, n, D, generator=g) * 0.1
    v = torch.randn(1, hkv, n, D, generator=g)
    k[:, :, 0] = 18.0 / (1.4426950408889634 * np.sqrt(D))
    v[:, :, 0] = 0.0
    q = (1.0 + 0.05 * torch.randn(b, hq, D, generator=g)).half().cuda()
    cache = wq.kv_quantize_keys(k.cuda()), wq.kv_quantize_values(v.cuda())
    full = [tuple(t.repeat(b, *[1] * (t.dim() - 1)) for t in part) for part in cache]
    got = wq.wq_prefix_attention(q, None, None, *full,
                                 torch.full((b,), n, dtype=torch.int32, device="cuda"))
    got, qn = got.double().cpu().numpy(), q.double().cpu().numpy()
    kk, vv = _rows(cache[0], False)[0], _rows(cache[1], True)[0]
    error = limit = 0.0
    for h in range(hkv):
        _, p, want = _attend(qn[:, h], kk[0, h], vv[0, h])
        step = 2.0 ** np.maximum(np.floor(np.log2(np.abs(want))) - 10, -24)
        error += ((got[:, h] - want) ** 2).sum()
        limit += (step ** 2 / 12).sum() + 2.0 ** -20 / 12 * (p ** 2 @ vv[0, h] ** 2).sum()
    assert error <= 1.05 ** 2 * limit, (error / limit) ** 0.5

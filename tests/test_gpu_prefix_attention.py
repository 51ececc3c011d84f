"""Decode attention over a shared prefix and each sequence's own tokens, against
the fp64 oracle.

Error bound of an output element. With p_l the exact weights (they sum to 1) and
A = sum_l p_l |v_l|:
  values   v is rounded to fp16 where the tensor cores of the prefix take it
           (2^-11 of itself; exact integers elsewhere), a weight is rounded to
           fp16 (2^-11, where it is at least 2^-14 of the largest; the weights
           below that are off by 2^-25 of the largest each): 2 * 2^-11 A, and
           2^-25 n A', A' the largest |v| and n the number of keys;
  scores   a key is rounded to fp16 as well: a score s_l = q . k_l / sqrt(D) is
           off by d_l <= 2^-11 sum_d |q_d k_ld| / sqrt(D), plus the fp32 sum of
           128 products and a few roundings of t: (128 * 2^-24) of the same sum
           and 2^-21 max(|s_l|, 24). A weight off by a factor e^d_l moves the
           numerator by sum_l p_l |v_l| (e^d_l - 1) and the denominator by
           sum_l p_l (e^d_l - 1);
  ex2      2^-22 a weight, in both sums: 2^-20 A with the fp32 sums' own.
Then the output's own half step.
"""

import numpy as np
import pytest
import torch

from oracle import kvcache

pytestmark = pytest.mark.gpu

D = 128


@pytest.fixture(scope="module")
def wq():
    from bit_weight_quantized_weights_b200 import binding
    return binding


@pytest.fixture(autouse=True, params=[0, 1, 2], ids=["auto", "mma", "tcgen05"])
def path(wq, request):
    """Every test on the chosen kernel and on both."""
    wq.wq_test_set_prefix_path(request.param)
    yield request.param
    wq.wq_test_set_prefix_path(0)


def _cache(wq, b, h, cap, seed, k_scale=0.5, v_scale=1.0):
    """(device K, device V, host K, host V) of quantized Gaussian rows."""
    g = torch.Generator().manual_seed(seed)
    dev, host = [], []
    for scale, quant in ((k_scale, wq.kv_quantize_keys), (v_scale, wq.kv_quantize_values)):
        x = torch.randn(b, h, cap, D, generator=g) * scale
        if quant is wq.kv_quantize_keys:
            x[..., 3] *= 8.0
        dev.append(quant(x.cuda()))
        q, s, z = dev[-1]
        w = q.cpu().numpy().view(np.uint32)
        if quant is wq.kv_quantize_keys:
            codes = np.stack([(w >> np.uint32(4 * i)) & 15 for i in range(8)], -1).reshape(
                b, h, cap, D)
        else:
            codes = np.stack([(w >> np.uint32(4 * i)) & 15 for i in range(8)], 3).reshape(
                b, h, -1, D)[:, :, :cap]
        host.append((codes, s.cpu().numpy(), z.cpu().numpy()))
    return dev + host


def _i32(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def _check(out, q, pk, pv, k, v, lengths, prefix_len, smallest=0.0):
    qn = q.double().cpu().numpy()
    want = kvcache.prefix_attention(qn, pk, pv, k, v, lengths, prefix_len)
    b_, hq, d = qn.shape
    hkv = k[0].shape[1]
    r = hq // hkv
    slack = np.zeros_like(want)
    for h in range(hkv):
        for b in range(b_):
            rows = [np.concatenate([_rows_of(pre, 0, h, prefix_len), _rows_of(own, b, h, lengths[b])])
                    for pre, own in ((pk, k), (pv, v))]
            kk, vv = rows[0], np.abs(rows[1])
            if len(kk) == 0:
                continue
            x = qn[b, h * r:(h + 1) * r]
            s = x @ kk.T / np.sqrt(d)
            p = np.exp(s - s.max(axis=1, keepdims=True))
            p /= p.sum(axis=1, keepdims=True)
            mag = np.abs(x) @ np.abs(kk).T / np.sqrt(d)
            delta = np.expm1(mag * (2.0 ** -11 + 2.0 ** -17)
                             + 2.0 ** -21 * np.maximum(np.abs(s), 24.0))
            o = np.abs(want[b, h * r:(h + 1) * r])
            a = p @ vv
            slack[b, h * r:(h + 1) * r] = (
                (2 * 2.0 ** -11 + 2.0 ** -20) * a + 2.0 ** -25 * len(kk) * vv.max()
                * p.max(axis=1, keepdims=True)
                + (p * delta) @ vv + o * (p * delta).sum(axis=1, keepdims=True))
    half = torch.finfo(out.dtype).eps / 2
    got = out.double().cpu().numpy()
    bound = slack + half * (np.abs(want) + slack) + 1e-30 + smallest
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), "%d elements off, worst %.2f of the bound" % (
        bad.sum(), float((np.abs(got - want) / bound).max()))
    # The roundings of many keys and dimensions are independent: as a whole the
    # error is near the output's own rounding (rms of a uniform error: half a
    # step / sqrt(3)); twice the half step leaves room for peaked rows.
    norm = np.linalg.norm(want)
    if out.numel() > 1000 and norm > 0:
        assert np.linalg.norm(got - want) <= (2 * half + 2.0 ** -10) * norm \
            + smallest * np.sqrt(want.size)


def _rows_of(cache, b, h, n):
    c, s, z = cache
    return (c[b, h, :n].astype(np.float64) - z[b, h, :n].astype(np.float64)[:, None]) * \
        s[b, h, :n].astype(np.float64)[:, None]


CASES = [
    # (B, Hq, Hkv, prefix, capacity, lengths)
    (1, 1, 1, 1, 1, [0]),
    (1, 1, 1, 1, 1, [1]),
    (1, 8, 8, 5, 3, [2]),
    (2, 2, 1, 33, 7, [7, 0]),
    (3, 8, 2, 100, 37, [0, 37, 5]),
    (2, 16, 2, 127, 130, [129, 64]),
    (5, 16, 1, 1000, 40, [0, 1, 40, 31, 32]),          # 80 prefix rows of one head
    (4, 12, 4, 515, 64, [8, 9, 63, 64]),               # R = 3
    (2, 14, 1, 301, 29, [29, 28]),                     # R = 14
    (9, 64, 8, 1025, 300, [300, 0, 1, 7, 8, 255, 256, 257, 299]),
    (17, 8, 1, 2049, 16, list(range(17))),             # 136 prefix rows
    (33, 8, 2, 513, 8, [i % 9 for i in range(33)]),
    (40, 8, 1, 777, 24, [i % 25 for i in range(40)]),  # 320 prefix rows
    (2, 8, 1, 5000, 4100, [4100, 3999]),               # several ranges of own tokens
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_matches_oracle(wq, case, dtype):
    b, hq, hkv, p, cap, lengths = case
    pk, pv, hpk, hpv = _cache(wq, 1, hkv, p, 1)
    k, v, hk, hv = _cache(wq, b, hkv, cap, 2)
    q = torch.randn(b, hq, D, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    out = wq.wq_prefix_attention(q, pk, pv, k, v, _i32(lengths))
    _check(out, q, hpk, hpv, hk, hv, lengths, p)


@pytest.mark.parametrize("b", [3, 40])
def test_prefix_shorter_than_its_cache_and_garbage_behind(wq, b):
    """Rows behind the prefix length and the sequences' lengths hold NaN scales
    and zeros and take no part; lengths outside 0 .. capacity are clamped."""
    hq, hkv, cap, p = 16, 2, 45, 301
    pk, pv, hpk, hpv = _cache(wq, 1, hkv, 333, 4)
    k, v, hk, hv = _cache(wq, b, hkv, cap, 5)
    lengths = [(7 * i) % (cap + 1) for i in range(b)]
    q = torch.randn(b, hq, D, generator=torch.Generator().manual_seed(6)).bfloat16().cuda()
    clean = wq.wq_prefix_attention(q, pk, pv, k, v, _i32(lengths), prefix_len=p)
    _check(clean, q, hpk, hpv, hk, hv, lengths, p)
    for part in (pk, pv):
        for t in part[1:]:
            t[:, :, p:] = float("nan")
    for part in (k, v):
        for t in part[1:]:
            for i, n in enumerate(lengths):
                t[i, :, n:] = float("inf") if i % 2 else float("nan")
    for part, n in ((pk, p),):
        part[0][:, :, n:] = -1
    dirty = wq.wq_prefix_attention(q, pk, pv, k, v, _i32(lengths), prefix_len=p)
    assert torch.equal(clean, dirty)
    far = [n if 0 < n < cap else (-5 if n == 0 else cap + 1000) for n in lengths]
    assert torch.equal(clean, wq.wq_prefix_attention(q, pk, pv, k, v, _i32(far), prefix_len=p))


def test_no_prefix_and_no_token(wq):
    """Without a prefix it is attention over each sequence's own tokens, and a
    sequence without any token gets zeros."""
    b, hq, hkv, cap = 4, 16, 2, 50
    k, v, hk, hv = _cache(wq, b, hkv, cap, 7)
    lengths = [0, 50, 1, 33]
    q = torch.randn(b, hq, D, generator=torch.Generator().manual_seed(8)).bfloat16().cuda()
    none = [(np.zeros((1, hkv, 0, D)), np.zeros((1, hkv, 0)), np.zeros((1, hkv, 0)))] * 2
    a = wq.wq_prefix_attention(q, None, None, k, v, _i32(lengths))
    _check(a, q, none[0], none[1], hk, hv, lengths, 0)
    assert not a[0].any()
    pk, pv, _, _ = _cache(wq, 1, hkv, 9, 9)
    assert torch.equal(a, wq.wq_prefix_attention(q, pk, pv, k, v, _i32(lengths), prefix_len=0))


@pytest.mark.parametrize("b", [2, 40])
def test_extreme_magnitudes(wq, b):
    """Queries from 2^-100 to 2^30, values whose rows span fp16's scales, and
    rows of zeros: every row keeps its own scaling."""
    hq, hkv, cap, p = 8, 1, 40, 200
    g = torch.Generator().manual_seed(10)
    pk, pv, hpk, hpv = _cache(wq, 1, hkv, p, 11, k_scale=1e-3, v_scale=1e-6)
    k, v, hk, hv = _cache(wq, b, hkv, cap, 12, k_scale=1e-3, v_scale=2e4)
    q = torch.randn(b, hq, D, generator=g)
    q[:, 0] *= 2.0 ** -100
    q[:, 1] *= 2.0 ** 12
    q[:, 2] = 0.0
    q[:, 3, 1:] *= 2.0 ** -20
    q = q.bfloat16().cuda()
    lengths = [cap - (i % 3) for i in range(b)]
    lengths[0] = 0                                       # only the tiny values of the prefix
    out = wq.wq_prefix_attention(q, pk, pv, k, v, _i32(lengths))
    _check(out, q, hpk, hpv, hk, hv, lengths, p)


@pytest.mark.parametrize("which", ["keys", "values"])
@pytest.mark.parametrize("scale", [5e-7, 2e-6, 1.5e-5, 1e-4])
def test_rows_whose_scales_are_subnormal(wq, scale, which):
    """fp16 scales of 3 to 650 times 2^-24: few keys, so that a row whose value
    is lost shows. Beyond the bound above, an fp16 output below 2^-14 is off by
    half of fp16's smallest number, 2^-25."""
    b, hq, p = 9, 16, 5
    g = torch.Generator().manual_seed(31)
    pk, pv, hpk, hpv = _cache(wq, 1, 1, p, 32, k_scale=scale if which == "keys" else 0.5,
                              v_scale=scale if which == "values" else 1.0)
    k, v, hk, hv = _cache(wq, b, 1, 8, 33)
    q = torch.randn(b, hq, D, generator=g)
    if which == "keys":
        q = (q * 2e4).clamp(-6e4, 6e4)
    q = q.half().cuda()
    lengths = [0] * b
    out = wq.wq_prefix_attention(q, pk, pv, k, v, _i32(lengths))
    _check(out, q, hpk, hpv, hk, hv, lengths, p, smallest=2.0 ** -25)


@pytest.mark.parametrize("b", [2, 40])
def test_sharp_and_growing_scores(wq, b):
    """Scores that grow along the keys (the running bound moves many times) and
    one key far above the rest."""
    hq, hkv, cap, p = 8, 1, 64, 600
    g = torch.Generator().manual_seed(13)
    x = torch.randn(1, hkv, p, D, generator=g) * 0.05
    x += torch.linspace(0, 4, p)[None, None, :, None]
    x[:, :, 77] += 3.0
    y = torch.randn(1, hkv, p, D, generator=g)
    pk, pv = wq.kv_quantize_keys(x.cuda()), wq.kv_quantize_values(y.cuda())

    def host(part, is_value):
        w = part[0].cpu().numpy().view(np.uint32)
        n = part[1].shape[2]
        c = np.stack([(w >> np.uint32(4 * i)) & 15 for i in range(8)], 3 if is_value else -1)
        return c.reshape(1, hkv, -1, D)[:, :, :n], part[1].cpu().numpy(), part[2].cpu().numpy()
    k, v, hk, hv = _cache(wq, b, hkv, cap, 14)
    q = (torch.randn(b, hq, D, generator=g) * 0.3 + 0.5).bfloat16().cuda()
    lengths = [cap] * b
    out = wq.wq_prefix_attention(q, pk, pv, k, v, _i32(lengths))
    _check(out, q, host(pk, False), host(pv, True), hk, hv, lengths, p)


@pytest.mark.parametrize("b", [3, 40])
def test_nan_query_stays_in_its_row(wq, b):
    hq, hkv, cap, p = 16, 2, 32, 150
    pk, pv, _, _ = _cache(wq, 1, hkv, p, 15)
    k, v, _, _ = _cache(wq, b, hkv, cap, 16)
    q = torch.randn(b, hq, D, generator=torch.Generator().manual_seed(17)).bfloat16().cuda()
    lengths = _i32([cap] * b)
    clean = wq.wq_prefix_attention(q, pk, pv, k, v, lengths)
    q[1, 3, 5] = float("nan")
    q[2, 9, 0] = float("inf")
    out = wq.wq_prefix_attention(q, pk, pv, k, v, lengths)
    assert bool(out[1, 3].isnan().all()) and not bool(out[2, 9].isfinite().any())
    out[1, 3], out[2, 9] = clean[1, 3], clean[2, 9]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("hq", [4, 16])
def test_sequences_do_not_depend_on_each_other(wq, hq):
    """A sequence's result is the same bits whatever the others hold."""
    b, hkv, cap, p = 24, 2, 70, 900
    pk, pv, _, _ = _cache(wq, 1, hkv, p, 18)
    k, v, _, _ = _cache(wq, b, hkv, cap, 19)
    k2, v2, _, _ = _cache(wq, b, hkv, cap, 20, k_scale=3.0, v_scale=50.0)
    q = torch.randn(b, hq, D, generator=torch.Generator().manual_seed(21)).bfloat16().cuda()
    a = wq.wq_prefix_attention(q, pk, pv, k, v, _i32([cap] * b))
    for part, other in zip(k + v, k2 + v2):
        other[5] = part[5]
    q2 = q.flip(0) * 7
    q2[5] = q[5]
    c = wq.wq_prefix_attention(q2, pk, pv, k2, v2, _i32([cap if i == 5 else 3 for i in range(b)]))
    assert torch.equal(a[5], c[5])


def test_fused_query_slice_streams_and_repeat(wq):
    """q as a slice of a fused projection; another stream; the same bits twice."""
    b, hq, hkv, cap, p = 20, 16, 2, 33, 400
    pk, pv, hpk, hpv = _cache(wq, 1, hkv, p, 22)
    k, v, hk, hv = _cache(wq, b, hkv, cap, 23)
    fused = torch.randn(b, hq + 2 * hkv, D,
                        generator=torch.Generator().manual_seed(24)).bfloat16().cuda()
    q = fused[:, :hq]
    lengths = [i % 34 for i in range(b)]
    out = wq.wq_prefix_attention(q, pk, pv, k, v, _i32(lengths))
    _check(out, q, hpk, hpv, hk, hv, lengths, p)
    ln = _i32(lengths)
    ws = wq.prefix_attention_workspace(b, hq, hkv, p, cap)
    ws.fill_(255)
    again = torch.empty_like(out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    wq.wq_prefix_attention(q, pk, pv, k, v, ln, workspace=ws, out=again, stream=side)
    side.synchronize()
    assert torch.equal(out, again)


def test_captured(wq):
    b, hq, hkv, cap, p = 18, 16, 2, 40, 300
    pk, pv, hpk, hpv = _cache(wq, 1, hkv, p, 25)
    k, v, hk, hv = _cache(wq, b, hkv, cap, 26)
    q = torch.randn(b, hq, D, generator=torch.Generator().manual_seed(27)).bfloat16().cuda()
    ln = _i32([1] * b)
    ws = wq.prefix_attention_workspace(b, hq, hkv, p, cap)
    out = wq.wq_prefix_attention(q, pk, pv, k, v, ln, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        wq.wq_prefix_attention(q, pk, pv, k, v, ln, workspace=ws, out=out)
    for lengths in ([40] * b, [0] * b, list(range(b))):
        q.copy_(torch.randn(b, hq, D).bfloat16())
        ln.copy_(_i32(lengths))
        graph.replay()
        _check(out, q, hpk, hpv, hk, hv, lengths, p)


def test_refusals(wq):
    b, hq, hkv, cap, p = 2, 8, 2, 16, 24
    pk, pv, _, _ = _cache(wq, 1, hkv, p, 28)
    k, v, _, _ = _cache(wq, b, hkv, cap, 29)
    q = torch.randn(b, hq, D).bfloat16().cuda()
    ln = _i32([1, 2])
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(q=q[:1]), dict(q=q.transpose(0, 1)),
                dict(ln=ln.long()), dict(ln=ln[:1]), dict(pk=k), dict(pk=None), dict(k=pk)):
        a = dict(q=q, pk=pk, pv=pv, k=k, v=v, ln=ln)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            wq.wq_prefix_attention(a["q"], a["pk"], a["pv"], a["k"], a["v"], a["ln"])
    with pytest.raises(wq.WqError):
        wq.wq_prefix_attention(q, pk, pv, k, v, ln, prefix_len=p + 1)
    with pytest.raises(wq.WqError):
        wq.wq_prefix_attention(q, pk, pv, k, v, ln,
                               workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(wq.WqError):                      # 9 heads over 2
        wq.wq_prefix_attention(torch.zeros(b, 9, D, dtype=torch.bfloat16, device="cuda"), pk, pv, k,
                               v, ln)


@pytest.mark.parametrize("b", [8, 40])  # 64 and 320 query rows: one and two row tiles
def test_bounded_wait_expires_cleanly(wq, b):
    """With the first key tile withheld the tensor-core kernel gives up, reports
    the wait and returns; the next call is right."""
    wq.wq_test_set_prefix_path(2)
    hq, hkv, cap, p = 8, 1, 16, 700
    pk, pv, hpk, hpv = _cache(wq, 1, hkv, p, 30)
    k, v, hk, hv = _cache(wq, b, hkv, cap, 31)
    q = torch.randn(b, hq, D, generator=torch.Generator().manual_seed(32)).bfloat16().cuda()
    ln = _i32([cap] * b)
    torch.cuda.synchronize()
    wq.wq_test_set_wait(1_000_000, 1)
    try:
        wq.wq_prefix_attention(q, pk, pv, k, v, ln)
        st, detail = wq.wq_device_error()
    finally:
        wq.wq_test_set_wait()
    assert st == wq.WQ_ERR_TIMEOUT and detail >> 8 in (0x41, 0x42, 0x43)
    assert wq.wq_device_error()[0] == wq.WQ_OK
    _check(wq.wq_prefix_attention(q, pk, pv, k, v, ln), q, hpk, hpv, hk, hv, [cap] * b, p)

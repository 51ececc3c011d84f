"""Caches and matrices whose element offsets pass 32 bits: token append and
read, prefix attention, MXFP4 planes and product."""

import pytest
import torch

pytestmark = pytest.mark.gpu

D = 128


@pytest.fixture(scope="module")
def wq():
    from bit_weight_quantized_weights_b200 import binding
    return binding


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def test_cache_rows_beyond_2_31_words(wq):
    """The third sequence of this cache starts at word 2^31 of the codes."""
    b, cap = 3, 2 ** 26 + 8
    k_cache, v_cache = wq.kv_cache_alloc(b, 1, cap)
    small = wq.kv_cache_alloc(b, 1, 64)
    g = torch.Generator().manual_seed(1)
    counts, starts = [3, 11, 40], [cap - 3, 2 ** 26 - 5, cap - 40]
    edges = [0, 3, 14, 54]
    k, v = (torch.randn(54, 1, D, generator=g).bfloat16().cuda() for _ in range(2))
    wq.wq_kv_append(k, v, k_cache, v_cache, _i32(starts), _i32(edges))
    wq.wq_kv_append(k, v, *small, _i32([s % 8 for s in starts]), _i32(edges))
    got = wq.wq_kv_read(k_cache, v_cache, _i32(starts), _i32(edges), 54)
    want = wq.wq_kv_read(*small, _i32([s % 8 for s in starts]), _i32(edges), 54)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (got[0].float() - k.float()).abs().max() < 0.5  # a step of 15 over a row's range
    assert int(torch.count_nonzero(k_cache[1])) == sum(counts)

    # attention of the first tokens of every sequence, the same rows in both caches
    zero = [0] * b
    wq.wq_kv_append(k, v, k_cache, v_cache, _i32(zero), _i32(edges))
    wq.wq_kv_append(k, v, *small, _i32(zero), _i32(edges))
    q = torch.randn(b, 4, D, generator=g).bfloat16().cuda()
    one = wq.wq_prefix_attention(q, None, None, k_cache, v_cache, _i32(counts))
    two = wq.wq_prefix_attention(q, None, None, *small, _i32(counts))
    # other key ranges: the weights' fp16 roundings differ (2^-11 of values up to
    # 4, on either side), and the outputs by a bf16 step
    assert torch.allclose(one.float(), two.float(), rtol=2.0 ** -7, atol=2.0 ** -8)


@pytest.mark.parametrize("b", [1, 20])  # 8 and 160 query rows
@pytest.mark.parametrize("path", [1, 2])
def test_prefix_of_2_27_tokens(wq, b, path):
    """Three keys at the far end decide: every other key scores 0, these 40 and
    more (each of the 2^27 others then weighs below 2^-57 of them)."""
    p, n = 2 ** 27 + 21, 3
    pk, pv = wq.kv_cache_alloc(1, 1, p)
    for part in (pk, pv):
        part[1].fill_(1.0)  # codes and zeros are 0: rows of zeros
    g = torch.Generator().manual_seed(2)
    k = torch.full((n, 1, D), 4.0)
    k[:, 0, 0] = torch.tensor([2.0, 3.0, 1.0])
    v = torch.randn(n, 1, D, generator=g)
    wq.wq_kv_append(k.cuda(), v.cuda(), pk, pv, _i32([p - n]), _i32([0, n]))
    q = torch.ones(b, 8, D, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 3.0
    kc, vc = wq.kv_cache_alloc(b, 1, 8)
    wq.wq_test_set_prefix_path(path)
    try:
        out = wq.wq_prefix_attention(q, pk, pv, kc, vc, _i32([0] * b))
        st, detail = wq.wq_device_error()
    finally:
        wq.wq_test_set_prefix_path(0)
    assert st == wq.WQ_OK, hex(detail)
    kr, vr = (t.double() for t in wq.wq_kv_read(pk, pv, _i32([p - n]), _i32([0, n]), n,
                                                dtype=torch.float32))
    s = q[0, :1].double() @ kr[:, 0].T / D ** 0.5
    want = torch.softmax(s, dim=-1) @ vr[:, 0]
    # keys and values rounded to fp16, weights too: 2^-11 each, the scores'
    # 2^-11 of about 46 and the bf16 output's half step
    bound = (3 * 2.0 ** -11 + 2 * 2.0 ** -11 * 46) * vr.abs().max() + 2.0 ** -8 * want.abs()
    assert ((out.double() - want).abs() <= bound).all()
    assert torch.equal(out, out[:1, :1].expand_as(out))


def test_planes_beyond_2_31_elements(wq):
    m, k = 2 ** 16 + 3, 2 ** 15 + 64
    x = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(3)
    rows = [0, 2 ** 15, m - 2, m - 1]
    x[rows] = torch.randn(4, k, generator=g).bfloat16().cuda()
    codes, scales = wq.wq_mx_quantize_planes(x, 2)
    want, ws = wq.wq_mx_quantize_planes(x[rows].contiguous(), 2)
    assert torch.equal(codes[:, rows], want) and torch.equal(scales[:, rows], ws)


def test_product_beyond_2_31_elements(wq):
    m, n, k = 2 ** 16 + 5, 2 ** 15 + 48, 128
    g = torch.Generator().manual_seed(4)
    rows = [0, 1, 2 ** 16 - 1, m - 2, m - 1]
    x = torch.randn(5, k, generator=g).bfloat16().cuda()
    wc, ws = wq.wq_mx_quantize((torch.randn(n, k, generator=g) * 0.02).cuda())
    big = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
    big[rows] = x
    y = wq.wq_mx_gemm(*wq.wq_mx_quantize_planes(big, 2), n, wc, ws)
    # exact block products, 8 of them added in fp32: the order may differ, by
    # 2 * 8 * 2^-23 of sum |x w| (about 1.6) and a bf16 step
    want = wq.wq_mx_gemm(*wq.wq_mx_quantize_planes(x, 2), n, wc, ws)
    assert torch.allclose(y[rows].float(), want.float(), rtol=2.0 ** -7, atol=4e-6)
    assert int(torch.count_nonzero(y)) == int(torch.count_nonzero(y[rows]))

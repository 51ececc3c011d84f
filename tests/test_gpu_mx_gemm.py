"""MXFP4 planes (bit for bit) and their product with MXFP4 weights for any M.

Error bound of an output: a block product (32 terms of E2M1 x E2M1 with two
power-of-two scales) is exact in fp32; the K / 32 block sums of every plane
are added in fp32, so the sum is within n 2^-23 sum |x| |w| of the exact one
for n = P K / 32 additions, whatever their order and whether the tensor core
rounds or truncates (2^-23), and the output is rounded once to bf16 (half an ulp).
"""

import numpy as np
import pytest
import torch

from oracle import mx

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def wq():
    from bit_weight_quantized_weights_b200 import binding
    return binding


def _x(m, k, dtype="bf16", seed=0):
    g = torch.Generator().manual_seed(100 + seed)
    x = torch.randn(m, k, generator=g)
    x[:, torch.randperm(k, generator=g)[:max(1, k // 100)]] *= 20.0
    return x.to(DTYPES[dtype])


def _pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _planes(x, n):
    """Oracle planes of fp64 x: packed codes, scale bytes, exact sum of planes."""
    c, s, hat = mx.mxfp4_two_pass(x)
    if n == 1:
        hat = mx.mx_dequant(c[0], s[0], "fp4")
    return (np.stack([_pack(v) for v in c[:n]]), np.stack(s[:n]), hat)


def _weights(wq, n, k, seed=0):
    g = torch.Generator().manual_seed(7 + seed)
    w = torch.randn(n, k, generator=g) * 0.02
    codes, scales = wq.wq_mx_quantize(w.cuda())
    c, s = mx.mx_quantize(w.double().numpy(), "fp4")
    assert np.array_equal(codes.cpu().numpy(), _pack(c)) and \
        np.array_equal(scales.cpu().numpy(), s)
    return codes, scales, mx.mx_dequant(c, s, "fp4")


def _check(y, hat, w, planes):
    want = hat @ w.T
    bound = planes * hat.shape[1] / 32 * 2.0 ** -23 * (np.abs(hat) @ np.abs(w).T)
    bound = bound + 2.0 ** -8 * (np.abs(want) + bound) + 1e-30
    got = y.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), "%d of %d off, worst %.2f of the bound, first at %s" % (
        bad.sum(), bad.size, float((np.abs(got - want) / bound).max()), np.argwhere(bad)[0])


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("m,k", [(1, 32), (3, 96), (5, 256), (2, 288), (33, 640), (130, 2048)])
def test_planes_bit_exact(wq, m, k, dtype):
    x = _x(m, k, dtype)
    for n in (1, 2):
        codes, scales, _ = _planes(x.double().numpy(), n)
        got, s = wq.wq_mx_quantize_planes(x.cuda(), n)
        assert np.array_equal(s.cpu().numpy(), scales)
        assert np.array_equal(got.cpu().numpy(), codes)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_planes_of_special_blocks(wq, dtype):
    """Zeros, negative zeros, halfway values, powers of two, the range's ends,
    subnormals, and elements 2^-120 of their block's largest."""
    rows = torch.zeros(12, 32)
    rows[1] = -0.0
    rows[2] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4)
    rows[3] = -rows[2]
    rows[4] = 2.0 ** torch.arange(-16, 16).float()
    rows[5, 3] = 3.0e38
    rows[6, 9] = 2.0 ** -126
    rows[7, 1] = 2.0 ** -133                             # subnormal
    rows[8, 0], rows[8, 1:] = 4.0, 2.0 ** -118
    rows[9, 0], rows[9, 5] = 2.0 ** 100, 2.0 ** -110
    rows[10] = 6.0 * 2.0 ** -3
    rows[11] = torch.linspace(-7, 7, 32)
    x = rows.to(DTYPES[dtype])
    codes, scales, _ = _planes(x.double().numpy(), 2)
    got, s = wq.wq_mx_quantize_planes(x.cuda(), 2)
    assert np.array_equal(s.cpu().numpy(), scales)
    assert np.array_equal(got.cpu().numpy(), codes)


def test_planes_match_the_byte_decomposition(wq):
    """The values are those of wq_mx_decompose (E4M3 bytes), and rows may be strided."""
    x = _x(9, 512).cuda()
    wide = torch.cat([x, x * 3], dim=1)
    planes, scales = wq.wq_mx_quantize_planes(wide[:, 512:], 2)
    ref, ref_s = wq.wq_mx_decompose((x * 3).contiguous(), 2)
    assert torch.equal(scales, ref_s)
    both = torch.stack([planes & 15, planes >> 4], -1).view(2, 9, 512).cpu().numpy()
    assert np.array_equal(mx.e2m1_decode(both), mx.e4m3_decode(ref.cpu().numpy()))


SHAPES = [
    # (M, N, K): one token, ragged tokens and features, K ending inside a stage
    (1, 16, 128), (1, 128, 256), (7, 48, 384), (16, 64, 512), (33, 80, 640), (127, 256, 256),
    (128, 256, 1024), (129, 272, 896), (200, 512, 2048), (300, 144, 1152), (513, 784, 512),
    (1, 4096, 4096), (40, 11008, 256), (1000, 2064, 384),
]


@pytest.mark.parametrize("planes", [1, 2])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(wq, m, n, k, planes):
    x = _x(m, k, seed=m)
    codes, scales, w = _weights(wq, n, k)
    _, _, hat = _planes(x.double().numpy(), planes)
    xc, xs = wq.wq_mx_quantize_planes(x.cuda(), planes)
    y = wq.wq_mx_gemm(xc, xs, n, codes, scales)
    st, detail = wq.wq_device_error()
    assert st == wq.WQ_OK, hex(detail)
    _check(y, hat, w, planes)


# Around the rule for scales taken without a pass: few rows, a tile a CTA, K past
# the ring of stages, K % 256 = 128, the last tile of features cut.
EDGES = [(20, 4736, 1152), (20, 4752, 1152), (72, 1040, 2176), (73, 1040, 2176), (128, 528, 4352),
         (144, 2048, 640), (160, 80, 4224)]


# Few tiles and a long K: two and four CTAs share it, its stages dividing and not,
# rows and features cut inside a tile, one and several row tiles.
SHARED = [(1, 4096, 4096), (33, 4080, 4224), (5, 1040, 8192), (128, 1024, 8320), (130, 2048, 8192),
          (400, 1040, 11008), (64, 2000, 2176)]


@pytest.mark.parametrize("planes", [1, 2])
@pytest.mark.parametrize("m,n,k", SHARED)
def test_product_whose_k_is_shared(wq, m, n, k, planes):
    test_product(wq, m, n, k, planes)


@pytest.mark.parametrize("planes", [1, 2])
@pytest.mark.parametrize("m,n,k", EDGES)
def test_product_with_and_without_the_scale_pass(wq, m, n, k, planes):
    test_product(wq, m, n, k, planes)


@pytest.mark.parametrize("m", [64, 400])
def test_every_code_and_scale_lands(wq, m):
    """Random codes and widely spread scale bytes: a scale taken for the wrong
    row or block is off by powers of two."""
    n, k = 272, 768
    r = np.random.RandomState(m)
    xc = r.randint(0, 256, (2, m, k // 2)).astype(np.uint8)
    xs = r.randint(97, 158, (2, m, k // 32)).astype(np.uint8)
    wc = r.randint(0, 256, (n, k // 2)).astype(np.uint8)
    ws = r.randint(97, 158, (n, k // 32)).astype(np.uint8)

    def value(c, s):
        both = np.stack([c & 15, c >> 4], -1).reshape(c.shape[:-1] + (-1,))
        return mx.mx_dequant(both, s, "fp4")
    y = wq.wq_mx_gemm(*[torch.from_numpy(t).cuda() for t in (xc, xs)], n,
                      *[torch.from_numpy(t).cuda() for t in (wc, ws)])
    hat, w = value(xc, xs), value(wc, ws)
    want = hat[0] @ w.T + hat[1] @ w.T
    mag = (np.abs(hat[0]) + np.abs(hat[1])) @ np.abs(w).T
    bound = 2 * k / 32 * 2.0 ** -23 * mag
    bound = bound + 2.0 ** -8 * (np.abs(want) + bound)
    assert (np.abs(y.double().cpu().numpy() - want) <= bound).all()


def test_many_tiles_and_repeat(wq):
    """More tiles than SMs, ragged on both sides; the same bits twice; rows of y
    around the written ones stay as they were."""
    m, n, k = 2500, 6160, 384
    x = _x(m, k, seed=5)
    codes, scales, w = _weights(wq, n, k, seed=1)
    _, _, hat = _planes(x.double().numpy(), 2)
    xc, xs = wq.wq_mx_quantize_planes(x.cuda(), 2)
    buf = torch.full((m + 2, n), 9.0, dtype=torch.bfloat16, device="cuda")
    y = wq.wq_mx_gemm(xc, xs, n, codes, scales, out=buf[1:-1])
    _check(y, hat, w, 2)
    assert bool((buf[0] == 9).all()) and bool((buf[-1] == 9).all())
    assert torch.equal(y, wq.wq_mx_gemm(xc, xs, n, codes, scales))


def test_captured_and_other_stream(wq):
    m, n, k = 70, 512, 1024
    codes, scales, w = _weights(wq, n, k)
    x = _x(m, k).cuda()
    planes, ps = wq.wq_mx_quantize_planes(x, 2)
    ws = wq.mx_gemm_workspace(m, n, k, 2)
    y = wq.wq_mx_gemm(planes, ps, n, codes, scales, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        wq.wq_mx_quantize_planes(x, 2, planes=planes, scales=ps)
        wq.wq_mx_gemm(planes, ps, n, codes, scales, workspace=ws, out=y)
    for seed in (21, 22):
        nx = _x(m, k, seed=seed)
        x.copy_(nx)
        graph.replay()
        _check(y, _planes(nx.double().numpy(), 2)[2], w, 2)


def test_empty_and_refusals(wq):
    codes, scales, _ = _weights(wq, 32, 256)
    x = _x(4, 256).cuda()
    p, s = wq.wq_mx_quantize_planes(x, 2)
    assert wq.wq_mx_gemm(p[:, :0].contiguous(), s[:, :0].contiguous(), 32, codes,
                         scales).shape == (0, 32)
    for call in (lambda: wq.wq_mx_quantize_planes(x.cpu(), 2),
                 lambda: wq.wq_mx_quantize_planes(x.t(), 2),
                 lambda: wq.wq_mx_quantize_planes(x.int(), 2),
                 lambda: wq.wq_mx_quantize_planes(x, 2, planes=p[:1]),
                 lambda: wq.wq_mx_gemm(p, s[:, :3], 32, codes, scales),
                 lambda: wq.wq_mx_gemm(p, s, 16, codes, scales),
                 lambda: wq.wq_mx_gemm(p.int(), s, 32, codes, scales),
                 lambda: wq.wq_mx_gemm(p, s, 32, codes, scales, out=x)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(wq.WqError):
        wq.wq_mx_quantize_planes(x, 3)
    with pytest.raises(wq.WqError):                      # rows 8 bytes apart from alignment
        wq.wq_mx_quantize_planes(torch.zeros(4, 260, dtype=torch.bfloat16,
                                             device="cuda")[:, :256], 1)
    p3, s3 = wq.wq_mx_quantize_planes(_x(4, 96).cuda(), 1)
    with pytest.raises(wq.WqError):                      # K % 128
        wq.wq_mx_gemm(p3, s3, 32, codes[:, :48].contiguous(), scales[:, :3].contiguous())


@pytest.mark.parametrize("m,n,k", [(200, 512, 1024), (20, 512, 1152), (20, 2048, 8192)])
def test_bounded_wait_expires_cleanly(wq, m, n, k):
    """With the loader's first k-tile withheld the kernel gives up, reports the
    wait and returns; the next call is right."""
    x = _x(m, k)
    codes, scales, w = _weights(wq, n, k)
    xc, xs = wq.wq_mx_quantize_planes(x.cuda(), 2)
    torch.cuda.synchronize()
    wq.wq_test_set_wait(1_000_000, 1)
    try:
        wq.wq_mx_gemm(xc, xs, n, codes, scales)
        st, detail = wq.wq_device_error()
    finally:
        wq.wq_test_set_wait()
    assert st == wq.WQ_ERR_TIMEOUT and detail >> 8 in (0x31, 0x32, 0x33, 0x34)
    assert wq.wq_device_error()[0] == wq.WQ_OK
    _check(wq.wq_mx_gemm(xc, xs, n, codes, scales), _planes(x.double().numpy(), 2)[2], w, 2)

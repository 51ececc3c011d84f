"""INT4 cache rows at the ends of the types' ranges, bit for bit against the oracle."""

import numpy as np
import pytest
import torch

from oracle import kvcache
from tests.test_gpu_kvcache import DTYPES, Pair, _i32

pytestmark = pytest.mark.gpu

D = 128


@pytest.fixture(scope="module")
def wq():
    from bit_weight_quantized_weights_b200 import binding
    return binding


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_whose_scale_is_infinite(wq, dtype):
    """Finite rows with (max - min) / 15 beyond fp16, or max - min beyond fp32: scale
    infinite, zero point and codes 0, as the quantizer of the weights has it; the rows
    between them and their V words are not touched by it."""
    g = torch.Generator().manual_seed(12)
    x = torch.randn(11, 1, D, generator=g)
    x[0, 0, 3], x[0, 0, 90] = -491400.0, 491400.0        # 982800 / 15 = 65520: rounds up
    x[2, 0, 0] = 1e6
    x[3, 0, 127] = -1e6
    x[5] = torch.randn(D, generator=g) * 1e7
    x[6, 0, 8], x[6, 0, 9] = 3e38, -3e38
    x[7] = 3e38
    x[8] = -3.3e38
    x[10, 0, 1] = 982000.0                               # the largest scale: 65472 rounds to it
    rows = x.to(DTYPES[dtype]).cuda()
    c = Pair(wq, 1, 1, 16, 9)
    with np.errstate(all="ignore"):
        c.append(wq, rows, rows, [3], [0, 11])
    assert np.isinf(c.host[0][1]).sum() >= 6
    c.check()
    codes, scales, zeros = wq.wq_quantize_pack(wq.WQ_FMT_INT4_ASYM,
                                               rows.float().view(11, D).contiguous(), D)
    for got, want in zip(c.k, (codes, scales[:, 0], zeros[:, 0])):
        assert torch.equal(got[0, 0, 3:14], want)
    for out in DTYPES.values():
        with np.errstate(all="ignore"):
            for got, cache in zip(wq.wq_kv_read(c.k, c.v, _i32([3]), _i32([0, 11]), 11, dtype=out),
                                  c.host):
                want = torch.from_numpy(kvcache.read(cache, [3], [0, 11], 11)).to(out)
                assert torch.equal(got.cpu().isnan(), want.isnan())
                assert torch.equal(got.cpu().nan_to_num(7.0), want.nan_to_num(7.0))


def test_a_prefix_length_without_a_prefix_is_refused(wq):
    own = wq.kv_cache_alloc(2, 1, 8)
    q = torch.zeros(2, 4, D, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        wq.wq_prefix_attention(q, None, None, *own, _i32([1, 2]), prefix_len=5)
    for none in (None, 0):
        assert not wq.wq_prefix_attention(q, None, None, *own, _i32([0, 0]), prefix_len=none).any()


def test_offsets_that_decrease_leave_the_rows_around(wq):
    """Arrays that break the contract: the read-back's rows before and behind both outputs,
    and the cache's sequences around, keep their values."""
    h, t, cap = 2, 32, 16
    k_cache, v_cache = wq.kv_cache_alloc(5, h, cap)
    inner = [tuple(x[1:4] for x in part) for part in (k_cache, v_cache)]
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(t, h, D, generator=g).bfloat16().cuda() for _ in range(2))
    for starts, edges in (([0, 3, 9], [5, 2, 40, 7]), ([2 ** 31 - 1, -2 ** 31, 0], [0, 32, 1, 31]),
                          ([0, 0, 0], [-9, 4, 99, 1000]), ([-7, 4, 15], [32, 31, 30, -1])):
        wq.wq_kv_append(k, v, *inner, _i32(starts), _i32(edges))
        for dtype in DTYPES.values():
            outs = [torch.full((t + 2, h, D), 3.0, dtype=dtype, device="cuda") for _ in range(2)]
            wq.wq_kv_read(*inner, _i32(starts), _i32(edges), t, k_out=outs[0][1:-1],
                          v_out=outs[1][1:-1])
            for out in outs:
                assert bool((out[0] == 3).all()) and bool((out[-1] == 3).all())
    for x in k_cache + v_cache:
        assert not x[0].any() and not x[4].any()

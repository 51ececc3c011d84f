"""Order on the GPU: a call sees what the calls before it on its stream wrote, whichever
kernels start early."""

import pytest
import torch

pytestmark = pytest.mark.gpu

D = 128


@pytest.fixture(scope="module")
def wq():
    from bit_weight_quantized_weights_b200 import binding
    return binding


def _i32(values):
    return torch.tensor(list(values), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("m", [1, 16])
def test_a_gemv_over_the_cache_an_append_wrote(wq, m, captured):
    """One head's K rows are INT4 weights of group 128. The decode GEMV loads its weights
    before it waits for the kernel in front of it: behind an append it must load what the
    append wrote."""
    h, n = 8, 16384                                      # the append takes some 20 us
    g = torch.Generator().manual_seed(3)
    k_cache, v_cache = wq.kv_cache_alloc(1, h, n)
    rows = [torch.randn(n, h, D, generator=g).bfloat16().cuda() for _ in range(3)]
    x = torch.randn(m, D, generator=g).bfloat16().cuda()
    starts, offsets = _i32([0]), _i32([0, n])
    k = rows[0].clone()
    y = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")

    def gemv(head, out=None):
        codes, scales, zeros = (t[0, head] for t in k_cache)
        return wq.wq_w4a16_gemv(x, n, wq.WQ_FMT_INT4_ASYM, D, codes, scales.view(n, 1),
                                zeros.view(n, 1), out=out)

    def step(head):
        wq.wq_kv_append(k, rows[1], k_cache, v_cache, starts, offsets)
        gemv(head, y)

    heads = [0, h - 1]
    for head in heads:
        step(head)
        torch.cuda.synchronize()
        if captured:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                step(head)
        for i in range(12):
            k.copy_(rows[i % 3])
            torch.cuda.synchronize()
            if captured:
                graph.replay()
            else:
                step(head)
            torch.cuda.synchronize()
            assert torch.equal(y, gemv(head)), (head, i)
    assert wq.wq_device_error()[0] == wq.WQ_OK

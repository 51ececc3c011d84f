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


def _calls(wq):
    """(name, call of a stream, bytes of the workspace it makes for itself)."""
    g = torch.Generator().manual_seed(9)
    m, n, k = 16, 512, 1024
    x = torch.randn(m, k, generator=g).bfloat16().cuda()
    big = torch.randn(300, k, generator=g).bfloat16().cuda()
    w = (torch.randn(n, k, generator=g) * 0.02).cuda()
    int4, nf4 = wq.WQ_FMT_INT4_ASYM, wq.WQ_FMT_NF4
    q4 = wq.wq_quantize_pack(int4, w, 128)
    f4 = wq.wq_quantize_pack(nf4, w, 64)
    mx = wq.wq_mx_quantize(w)
    rt = wq.wq_residual(int4, w, 128, *q4)
    planes = wq.wq_mx_quantize_planes(big, 2)
    b, hq, hkv, cap, p = 24, 16, 2, 700, 900
    q = torch.randn(b, hq, D, generator=g).bfloat16().cuda()
    rows = [torch.randn(b, hkv, cap, D, generator=g).cuda() for _ in range(2)]
    own = wq.kv_quantize_keys(rows[0]), wq.kv_quantize_values(rows[1])
    pre = [torch.randn(1, hkv, p, D, generator=g).cuda() for _ in range(2)]
    pre = wq.kv_quantize_keys(pre[0]), wq.kv_quantize_values(pre[1])
    starts, offsets = _i32([0] * b), _i32(range(0, 100 * b + 1, 100))
    lengths = _i32([30 * i for i in range(b)])
    size = lambda op, rows_, c: wq.wq_workspace_bytes(op, rows_, n, k, 128, c)
    return [
        ("quantize_pack", lambda s: wq.wq_quantize_pack(int4, w, 128, stream=s)[:2], 0),
        ("unpack", lambda s: wq.wq_unpack(int4, q4[0], n, k, stream=s), 0),
        ("nf4_dequant", lambda s: wq.wq_nf4_dequant(*f4[:2], n * k, stream=s), 0),
        ("int4_dequant", lambda s: wq.wq_int4_dequant(*q4, n, k, 128, stream=s), 0),
        ("residual", lambda s: wq.wq_residual(int4, w, 128, *q4, stream=s), 0),
        ("gemv", lambda s: wq.wq_w4a16_gemv(x, n, int4, 128, *q4, stream=s), 0),
        ("salient", lambda s: wq.wq_w4a16_gemv_salient(x, n, int4, 128, *q4, rt, 64, stream=s), 256),
        ("gemm", lambda s: wq.wq_w4a16_gemm(big, n, int4, 128, *q4, stream=s),
         size(wq.WQ_OP_GEMM, 300, 1)),
        ("decompose", lambda s: wq.wq_msd_decompose(x, 2, stream=s), 0),
        ("msd", lambda s: wq.wq_msd_gemm(big, n, 2, 128, *q4, stream=s),
         size(wq.WQ_OP_MSD_GEMM, 300, 2)),
        ("msd decode", lambda s: wq.wq_msd_gemm(x, n, 2, 128, *q4, stream=s),
         size(wq.WQ_OP_MSD_GEMM, m, 2)),
        ("msd nf4", lambda s: wq.wq_msd_gemm_nf4(x, n, 2, *f4[:2], stream=s),
         size(wq.WQ_OP_MSD_GEMM, m, 2)),
        ("mx_quantize", lambda s: wq.wq_mx_quantize(w, stream=s), 0),
        ("mx_decompose", lambda s: wq.wq_mx_decompose(x, 2, stream=s), 0),
        ("mx_gemv", lambda s: wq.wq_mx_gemv(x, n, 2, *mx, stream=s), size(wq.WQ_OP_MX_GEMV, m, 2)),
        ("planes", lambda s: wq.wq_mx_quantize_planes(big, 2, stream=s), 0),
        ("mx_gemm", lambda s: wq.wq_mx_gemm(*planes, n, *mx, stream=s),
         size(wq.WQ_OP_MX_GEMM, 300, 2)),
        ("kv values", lambda s: wq.kv_quantize_values(rows[1], stream=s), 0),
        ("kv_read", lambda s: wq.wq_kv_read(*own, starts, offsets, 100 * b, stream=s), 0),
        ("prefix", lambda s: wq.wq_prefix_attention(q, *pre, *own, lengths, stream=s),
         wq.prefix_attention_workspace(b, hq, hkv, p, cap).numel()),
        ("attention", lambda s: wq.wq_msd_decode_attention(q, *own, stream=s),
         wq.attention_workspace(b, hq, hkv, cap, D, 2, "cuda").numel()),
    ]


NAMES = ["quantize_pack", "unpack", "nf4_dequant", "int4_dequant", "residual", "gemv", "salient",
         "gemm", "decompose", "msd", "msd decode", "msd nf4", "mx_quantize", "mx_decompose",
         "mx_gemv", "planes", "mx_gemm", "kv values", "kv_read", "prefix", "attention"]


@pytest.fixture(scope="module")
def calls(wq):
    found = {name: rest for name, *rest in _calls(wq)}
    assert sorted(found) == sorted(NAMES)
    return found


@pytest.mark.parametrize("name", NAMES)
def test_a_call_on_another_stream_owns_what_it_allocates(calls, name):
    """With stream= and no buffers given: what is allocated and freed on the current stream,
    before the call or right after it, is none of the call's memory."""
    call, scratch = calls[name]
    many = lambda out: out if isinstance(out, tuple) else (out,)
    want = [t.clone() for t in many(call(None))]
    sizes = sorted({scratch} | {t.nbytes for t in want} - {0})
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for wait in (4_000_000, 0):                          # the call begins late, or at once
        # blocks of these sizes, freed while a long kernel and then a fill are pending
        blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
        if not wait:
            torch.cuda._sleep(4_000_000)
        for t in blocks:
            t.fill_(255)
        del blocks, t
        with torch.cuda.stream(side):
            torch.cuda._sleep(wait or 1)
        got = many(call(side))
        # and blocks taken from the pool as soon as the call has returned
        taken = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
        for t in taken:
            t.fill_(255)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(bool((t == 255).all()) for t in taken)
        del got, taken, t

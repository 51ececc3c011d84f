"""The 4-bit serving operators as an attention block uses them: MXFP4 projections,
keys and values into the INT4 cache as they are written, attention over a shared
prefix, and the output projection; step by step, captured and replayed."""

import numpy as np
import pytest
import torch

from oracle import kvcache, mx

pytestmark = pytest.mark.gpu

D = 128


@pytest.fixture(scope="module")
def wq():
    from bit_weight_quantized_weights_b200 import binding
    return binding


def _linear(x, w, planes):
    """fp64 product of MXFP4 planes of x with dequantized weights w."""
    c, s, hat = mx.mxfp4_two_pass(x)
    if planes == 1:
        hat = mx.mx_dequant(c[0], s[0], "fp4")
    return hat @ w.T, np.abs(hat) @ np.abs(w).T


def _close_bf16(got, want, slack):
    got = got.double().cpu().numpy()
    bound = slack + 2.0 ** -8 * (np.abs(want) + slack) + 1e-30
    assert (np.abs(got - want) <= bound).all(), float((np.abs(got - want) / bound).max())


@pytest.mark.parametrize("b,hq,hkv,planes", [(3, 8, 2, 2), (40, 8, 1, 1)])
def test_attention_block_decodes(wq, b, hq, hkv, planes):
    """Every stage of every step against fp64 from the stage's own inputs; the
    step is captured once and replayed with the positions kept on the GPU."""
    hidden, prefix, cap, steps = 384, 200, 24, 4
    g = torch.Generator().manual_seed(5)
    n_qkv = (hq + 2 * hkv) * D
    weights = []
    for n, k in ((n_qkv, hidden), (hidden, hq * D)):
        w = torch.randn(n, k, generator=g) * 0.05
        codes, scales = wq.wq_mx_quantize(w.cuda())
        weights.append((codes, scales, mx.mx_dequant(*mx.mx_quantize(w.double().numpy(), "fp4"),
                                                     "fp4")))
    pre = [torch.randn(1, hkv, prefix, D, generator=g) for _ in range(2)]
    pk, pv = wq.kv_quantize_keys(pre[0].cuda()), wq.kv_quantize_values(pre[1].cuda())
    kc, vc = wq.kv_cache_alloc(b, hkv, cap)

    x = torch.zeros(b, hidden, dtype=torch.bfloat16, device="cuda")
    first = [5 * (i % 3) for i in range(b)]              # ragged starts: earlier tokens are zeros
    starts = torch.tensor(first, dtype=torch.int32, device="cuda")
    lengths = torch.zeros(b, dtype=torch.int32, device="cuda")
    offsets = torch.arange(b + 1, dtype=torch.int32, device="cuda")
    qkv = torch.empty(b, n_qkv, dtype=torch.bfloat16, device="cuda")
    attn = torch.empty(b, hq, D, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(b, hidden, dtype=torch.bfloat16, device="cuda")
    ws1 = wq.mx_gemm_workspace(b, n_qkv, hidden, planes)
    ws2 = wq.prefix_attention_workspace(b, hq, hkv, prefix, cap)
    ws3 = wq.mx_gemm_workspace(b, hidden, hq * D, planes)

    def step():
        p, s = wq.wq_mx_quantize_planes(x, planes)
        wq.wq_mx_gemm(p, s, n_qkv, weights[0][0], weights[0][1], workspace=ws1, out=qkv)
        rows = qkv.view(b, hq + 2 * hkv, D)
        wq.wq_kv_append(rows[:, hq:hq + hkv], rows[:, hq + hkv:], kc, vc, starts, offsets)
        torch.add(starts, 1, out=lengths)
        wq.wq_prefix_attention(rows[:, :hq], pk, pv, kc, vc, lengths, workspace=ws2, out=attn)
        p, s = wq.wq_mx_quantize_planes(attn.view(b, hq * D), planes)
        wq.wq_mx_gemm(p, s, hidden, weights[1][0], weights[1][1], workspace=ws3, out=y)
        starts.add_(1)

    step()
    starts.copy_(torch.tensor(first, dtype=torch.int32))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    starts.copy_(torch.tensor(first, dtype=torch.int32))

    host = []
    for words, dev in ((kvcache.key_words, kc), (kvcache.value_words, vc)):
        host.append((np.zeros((b, hkv, cap, D), np.uint8), np.zeros((b, hkv, cap), np.float16),
                     np.zeros((b, hkv, cap), np.float16)))
        for t in dev:
            t.zero_()
    prefix_rows = []
    for part, is_value in ((pk, False), (pv, True)):
        w = part[0].cpu().numpy().view(np.uint32)
        c = np.stack([(w >> np.uint32(4 * i)) & 15 for i in range(8)], 3 if is_value else -1)
        prefix_rows.append((c.reshape(1, hkv, -1, D)[:, :, :prefix], part[1].cpu().numpy(),
                            part[2].cpu().numpy()))
    for i in range(steps):
        x.copy_(torch.randn(b, hidden, generator=g).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        # projection: fp32 sums of block products that are exact
        want, mag = _linear(x.double().cpu().numpy(), weights[0][2], planes)
        _close_bf16(qkv, want, planes * hidden / 32 * 2.0 ** -23 * mag)
        # cache: bit for bit from the projection's own output
        rows = qkv.view(b, hq + 2 * hkv, D).float().cpu().numpy()
        at = [f + i for f in first]
        edges = list(range(b + 1))
        kvcache.append(host[0], rows[:, hq:hq + hkv], at, edges)
        kvcache.append(host[1], rows[:, hq + hkv:], at, edges)
        for (codes, sc, zr), dev, words in zip(host, (kc, vc),
                                               (kvcache.key_words, kvcache.value_words)):
            assert np.array_equal(dev[0].cpu().numpy().view(np.uint32), words(codes))
            assert np.array_equal(dev[1].cpu().numpy(), sc)
            assert np.array_equal(dev[2].cpu().numpy(), zr)
        # attention over the prefix and what the cache holds (the skipped first
        # rows are rows of zero codes and scales: the values 0)
        lens = [p + 1 for p in at]
        want = kvcache.prefix_attention(rows[:, :hq], prefix_rows[0], prefix_rows[1], host[0],
                                        host[1], lens, prefix)
        got = attn.double().cpu().numpy()
        assert np.linalg.norm(got - want) <= 5e-3 * np.linalg.norm(want)
        assert np.abs(got - want).max() <= 2e-2 * np.abs(want).max()
        want, mag = _linear(attn.view(b, hq * D).double().cpu().numpy(), weights[1][2], planes)
        _close_bf16(y, want, planes * hq * D / 32 * 2.0 ** -23 * mag)
    assert wq.wq_device_error()[0] == wq.WQ_OK


def test_operators_on_two_streams_at_once(wq):
    """The same calls on two streams that run together, each with its own
    workspace and outputs, give what they give one after the other."""
    g = torch.Generator().manual_seed(21)
    b, hq, hkv, p, cap = 24, 16, 2, 3000, 40
    q = torch.randn(b, hq, D, generator=g).bfloat16().cuda()
    prompt, own = wq.kv_cache_alloc(1, hkv, p), wq.kv_cache_alloc(b, hkv, cap)
    rows = [torch.randn(n, hkv, D, generator=g).bfloat16().cuda() for n in (p, p, b * 30, b * 30)]
    i32 = lambda v: torch.tensor(list(v), dtype=torch.int32, device="cuda")
    wq.wq_kv_append(*rows[:2], *prompt, i32([0]), i32([0, p]))
    starts, edges, lengths = i32([0] * b), i32(range(0, 30 * b + 1, 30)), i32([30] * b)
    wq.wq_kv_append(*rows[2:], *own, starts, edges)
    x = torch.randn(300, 1024, generator=g).bfloat16().cuda()
    wc, ws = wq.wq_mx_quantize((torch.randn(2048, 1024, generator=g) * 0.02).cuda())

    def step(work):
        planes, scales = wq.wq_mx_quantize_planes(x, 2)
        y = wq.wq_mx_gemm(planes, scales, 2048, wc, ws, workspace=work[0])
        small = wq.wq_mx_gemm(planes[:, :20].contiguous(), scales[:, :20].contiguous(), 2048, wc,
                              ws, workspace=work[1])
        outs = []
        for path in (1, 2):
            wq.wq_test_set_prefix_path(path)
            outs.append(wq.wq_prefix_attention(q, *prompt, *own, lengths, workspace=work[2]))
        return [y, small, *outs, *wq.wq_kv_read(*own, starts, edges, 30 * b)]

    def workspaces():
        sizes = []
        for path in (1, 2):
            wq.wq_test_set_prefix_path(path)
            sizes.append(wq.prefix_attention_workspace(b, hq, hkv, p, cap).numel())
        return (wq.mx_gemm_workspace(300, 2048, 1024), wq.mx_gemm_workspace(20, 2048, 1024),
                torch.empty(max(sizes), dtype=torch.uint8, device="cuda"))

    try:
        work = [workspaces(), workspaces()]
        want = step(work[0])
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        got = [[], []]
        for _ in range(10):
            for i, stream in enumerate(streams):
                with torch.cuda.stream(stream):
                    got[i].append(step(work[i]))
        torch.cuda.synchronize()
    finally:
        wq.wq_test_set_prefix_path(0)
    assert wq.wq_device_error()[0] == wq.WQ_OK
    for outs in got[0] + got[1]:
        assert all(torch.equal(a, c) for a, c in zip(outs, want))


@pytest.mark.parametrize("path", [1, 2])
def test_a_chain_without_waits(wq, path):
    """Every call reads what the call before it wrote, with torch operations
    between some of them: the same results as with a synchronization after each."""
    b, hkv, cap, n = 16, 2, 70, 1024
    g = torch.Generator().manual_seed(5)
    x0 = torch.randn(b, n, generator=g).bfloat16().cuda()
    weights = [wq.wq_mx_quantize((torch.randn(n, n, generator=g) * 0.03).cuda()) for _ in range(2)]
    prompt = [torch.randn(200, hkv, D, generator=g).bfloat16().cuda() for _ in range(2)]
    i32 = lambda v: torch.tensor(list(v), dtype=torch.int32, device="cuda")
    edges, zero = i32(range(b + 1)), i32([0])

    def run(wait):
        pre, own = wq.kv_cache_alloc(1, hkv, 200), wq.kv_cache_alloc(b, hkv, cap)
        wq.wq_kv_append(*prompt, *pre, zero, i32([0, 200]))
        x, outs, starts = x0.clone(), [], i32([0] * b)
        for step in range(40):
            planes, scales = wq.wq_mx_quantize_planes(x, 2)
            wait()
            y = wq.wq_mx_gemm(planes, scales, n, *weights[0])
            wait()
            q = y.view(b, 8, D)
            wq.wq_kv_append(q[:, :2], q[:, 2:4], *own, starts, edges)
            wait()
            starts += 1
            o = wq.wq_prefix_attention(q, *pre, *own, starts)
            wait()
            k, v = wq.wq_kv_read(*own, starts - 1, edges, b)
            planes, scales = wq.wq_mx_quantize_planes(o.view(b, n), 1)
            wait()
            x = wq.wq_mx_gemm(planes, scales, n, *weights[1])
            wait()
            x = (x + x0).clamp(-4, 4)
            outs += [y, o, k, v, x]
        return outs

    wq.wq_test_set_prefix_path(path)
    try:
        want = run(torch.cuda.synchronize)
        for _ in range(3):
            assert all(torch.equal(a, c) for a, c in zip(run(lambda: None), want))
    finally:
        wq.wq_test_set_prefix_path(0)
    assert wq.wq_device_error()[0] == wq.WQ_OK

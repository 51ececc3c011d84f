"""INT4 KV cache: tokens appended at ragged positions and rows read back, bit
for bit against the oracle; the rows around stay as they were."""

import numpy as np
import pytest
import torch

from oracle import kvcache

pytestmark = pytest.mark.gpu

D = 128
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def wq():
    from bit_weight_quantized_weights_b200 import binding
    return binding


def _edges(counts):
    return [0] + [int(c) for c in np.cumsum(counts)]


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Pair:
    """The same cache on both sides: random content on the GPU, its unpacked rows here."""

    def __init__(self, wq, b, h, cap, seed):
        r = np.random.RandomState(seed)
        self.host, dev = [], []
        for words in (kvcache.key_words, kvcache.value_words):
            codes = r.randint(0, 16, (b, h, cap, D)).astype(np.uint8)
            s = (r.rand(b, h, cap) + 0.01).astype(np.float16)
            z = r.randint(0, 16, (b, h, cap)).astype(np.float16)
            self.host.append((codes, s, z))
            dev.append((torch.from_numpy(words(codes).view(np.int32)).cuda(),
                        torch.from_numpy(s).cuda(), torch.from_numpy(z).cuda()))
        self.k, self.v = dev

    def append(self, wq, k, v, starts, offsets):
        wq.wq_kv_append(k, v, self.k, self.v, _i32(starts), _i32(offsets))
        for cache, rows in zip(self.host, (k, v)):
            kvcache.append(cache, rows.float().cpu().numpy(), starts, offsets)

    def check(self):
        for (codes, s, z), dev, words in zip(self.host, (self.k, self.v),
                                             (kvcache.key_words, kvcache.value_words)):
            assert np.array_equal(dev[1].cpu().numpy().view(np.uint16), s.view(np.uint16))
            assert np.array_equal(dev[2].cpu().numpy(), z)
            got = dev[0].cpu().numpy().view(np.uint32)
            want = words(codes)
            assert np.array_equal(got, want)


def _rows(t, h, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(t, h, D, generator=g) * scale).to(DTYPES[dtype]).cuda() for _ in range(2)]


CASES = [
    # (heads, capacity, starts, counts)
    (1, 8, [0], [8]),                        # one whole block
    (2, 5, [0], [1]),                        # a capacity inside a block
    (3, 37, [3, 0, 36], [1, 0, 1]),          # single tokens, an empty sequence, the last row
    (2, 64, [5, 7, 8, 1, 0], [3, 17, 9, 0, 64]),
    (8, 100, [99, 0, 50, 13], [1, 100, 7, 30]),
    (1, 40, [0] * 70, [1] * 70),             # more sequences than a warp has lanes
    (2, 16, [1] * 33, [0, 5] * 16 + [9]),
    (1, 9, [0] * 1100, [1, 0, 2, 0] * 275),  # three levels of the search
]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_append_and_read_bit_exact(wq, case, dtype):
    h, cap, starts, counts = case
    c = Pair(wq, len(starts), h, cap, 3)
    edges = _edges(counts)
    k, v = _rows(edges[-1], h, dtype, 5)
    c.append(wq, k, v, starts, edges)
    c.check()
    for out in DTYPES.values():
        got = wq.wq_kv_read(c.k, c.v, _i32(starts), _i32(edges), edges[-1], dtype=out)
        for g, cache in zip(got, c.host):
            want = torch.from_numpy(kvcache.read(cache, starts, edges, edges[-1])).to(out)
            assert torch.equal(g.cpu(), want)


def test_matches_the_whole_cache_quantizer(wq):
    """Appending a cache token by token gives the cache quantized at once."""
    b, h, n = 2, 3, 21
    g = torch.Generator().manual_seed(8)
    k, v = [torch.randn(b, h, n, D, generator=g).cuda() for _ in range(2)]
    want = wq.kv_quantize_keys(k), wq.kv_quantize_values(v)
    kc, vc = wq.kv_cache_alloc(b, h, n)
    for t in range(n):
        wq.wq_kv_append(k[:, :, t], v[:, :, t], kc, vc, _i32([t] * b), _i32(range(b + 1)))
    for got, ref in zip(kc + vc, want[0] + want[1]):
        assert torch.equal(got, ref)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_strided_rows(wq, dtype):
    """Keys and values as slices of a fused projection, heads before tokens, and
    a read-back into slices of a larger tensor."""
    h, t = 4, 13
    g = torch.Generator().manual_seed(1)
    fused = torch.randn(t, 3 * h, D, generator=g).to(DTYPES[dtype]).cuda()
    head_first = torch.randn(h, t, D, generator=g).to(DTYPES[dtype]).cuda().transpose(0, 1)
    c = Pair(wq, 2, h, 24, 4)
    c.append(wq, fused[:, h:2 * h], head_first, [2, 9], [0, 6, 13])
    c.check()
    big = torch.full((t + 2, 2 * h, D), 7.0, dtype=DTYPES[dtype], device="cuda")
    wq.wq_kv_read(c.k, c.v, _i32([2, 9]), _i32([0, 6, 13]), t, k_out=big[1:-1, :h],
                  v_out=big[1:-1, h:])
    for part, cache in zip((big[1:-1, :h], big[1:-1, h:]), c.host):
        want = torch.from_numpy(kvcache.read(cache, [2, 9], [0, 6, 13], t)).to(DTYPES[dtype])
        assert torch.equal(part.cpu(), want)
    assert bool((big[0] == 7).all()) and bool((big[-1] == 7).all())


def test_one_token_or_head_of_any_stride(wq):
    """The stride of a dimension of one element means nothing."""
    h, cap = 2, 9
    g = torch.Generator().manual_seed(77)
    for shape in ((1, h), (3, 1)):
        x = torch.randn(shape[0], 2 * shape[1] * D + (4 if shape[0] == 1 else 0), generator=g)
        x = x.bfloat16().cuda()
        n = shape[1] * D
        k, v = (x[:, i * n:(i + 1) * n].unflatten(1, (shape[1], D)) for i in (0, 1))
        if shape[1] == 1:
            k, v = (t.as_strided(t.shape, (t.stride(0), 4, 1), t.storage_offset()) for t in (k, v))
        starts, offsets = _i32([1]), _i32([0, shape[0]])
        caches = [wq.kv_cache_alloc(1, shape[1], cap) for _ in range(2)]
        wq.wq_kv_append(k, v, *caches[0], starts, offsets)
        wq.wq_kv_append(k.contiguous(), v.contiguous(), *caches[1], starts, offsets)
        for a, b in zip(caches[0][0] + caches[0][1], caches[1][0] + caches[1][1]):
            assert torch.equal(a, b)


def test_values_on_rounding_borders(wq):
    """Rows of zeros, of one sign, of a single large value, subnormal ranges,
    halfway codes, and the largest finite bf16 that fits fp16 scales."""
    t = 12
    x = torch.zeros(t, 1, D)
    x[1] = 3.0
    x[2] = -2.5
    x[3, 0, 7] = 60000.0
    x[4] = torch.linspace(0, 15, D)[None]
    x[5] = torch.arange(D)[None] % 16 + 0.5
    x[6] = torch.randn(D, generator=torch.Generator().manual_seed(2)) * 1e-7
    x[7] = torch.randn(D, generator=torch.Generator().manual_seed(3)) * 1e-6
    x[8] = torch.randn(D, generator=torch.Generator().manual_seed(4)) * 3e4
    x[9, 0, 0], x[9, 0, 1] = -490000.0, 490000.0
    x[10, 0, 5] = 2.0 ** -126
    x[11] = torch.arange(D)[None] * 0.25 - 16
    for dtype in (torch.bfloat16, torch.float32):
        c = Pair(wq, 1, 1, 16, 9)
        rows = x.to(dtype).cuda()
        c.append(wq, rows, rows, [3], [0, t])
        c.check()


def test_positions_outside_and_rows_behind(wq):
    """Positions outside the capacity are dropped on append and read as zeros;
    rows behind the last sequence stay as they were."""
    c = Pair(wq, 3, 2, 20, 6)
    starts, edges = [-3, 17, 2000], [0, 5, 11, 13]
    k, v = _rows(16, 2, "bf16", 7)
    c.append(wq, k, v, starts, edges)
    c.check()
    ko = torch.full((16, 2, D), 5.0, dtype=torch.float32, device="cuda")
    vo = ko.clone()
    wq.wq_kv_read(c.k, c.v, _i32(starts), _i32(edges), 16, k_out=ko, v_out=vo)
    for got, cache in zip((ko, vo), c.host):
        want = kvcache.read(cache, starts, edges, 13)
        assert np.array_equal(got[:13].double().cpu().numpy(), want)
        assert bool((got[13:] == 5).all())


def test_offsets_that_decrease_stay_inside(wq):
    """Arrays that break the contract: no access outside the buffers (the
    guard rows around them keep their values)."""
    h, t, cap = 2, 32, 16
    kc, vc = wq.kv_cache_alloc(5, h, cap)
    inner = [tuple(x[1:4] for x in part) for part in (kc, vc)]
    k, v = _rows(t, h, "bf16", 2)
    for starts, edges in (([0, 3, 9], [5, 2, 40, 7]), ([2 ** 31 - 1, -2 ** 31, 0], [0, 32, 1, 31]),
                          ([0, 0, 0], [-9, 4, 99, 1000])):
        wq.wq_kv_append(k, v, *inner, _i32(starts), _i32(edges))
        out = torch.full((t + 2, h, D), 3.0, device="cuda")
        wq.wq_kv_read(*inner, _i32(starts), _i32(edges), t, k_out=out[1:-1], v_out=out[1:-1].clone())
        assert bool((out[0] == 3).all()) and bool((out[-1] == 3).all())
    for x in kc + vc:
        assert not x[0].any() and not x[4].any()


def test_empty_and_refusals(wq):
    kc, vc = wq.kv_cache_alloc(2, 2, 16)
    k, v = _rows(4, 2, "bf16", 1)
    s, o = _i32([0, 0]), _i32([0, 2, 4])
    wq.wq_kv_append(k[:0], v[:0], kc, vc, s, _i32([0, 0, 0]))
    assert wq.wq_kv_read(kc, vc, s, _i32([0, 0, 0]), 0)[0].shape == (0, 2, D)
    assert not kc[0].any() and not vc[0].any()
    for bad in (dict(k=k.cpu()), dict(k=k.half()), dict(k=k[:, :1]), dict(k=k[:3]), dict(s=s[:1]),
                dict(o=o.long()), dict(o=o[:2]), dict(kc=vc), dict(kc=kc[:2] + (kc[2][:1],)),
                dict(k=k.transpose(1, 2).contiguous().transpose(1, 2))):
        a = dict(k=k, v=v, kc=kc, vc=vc, s=s, o=o)
        a.update(bad)
        with pytest.raises(ValueError):
            wq.wq_kv_append(a["k"], a["v"], a["kc"], a["vc"], a["s"], a["o"])
    wide = torch.zeros(4, 2, D + 4, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(wq.WqError):                      # rows 264 bytes apart
        wq.wq_kv_append(wide[..., :D], v, kc, vc, s, o)
    with pytest.raises(wq.WqError):                      # rows that start 8 bytes in
        wq.wq_kv_append(k, torch.zeros(4 * 2 * D + 4, dtype=torch.bfloat16,
                                       device="cuda")[4:].view(4, 2, D), kc, vc, s, o)
    with pytest.raises(ValueError):
        wq.wq_kv_read(kc, vc, s, o, 5, k_out=k, v_out=v)


def test_captured_append_follows_the_arrays(wq):
    """A captured append and read-back replayed with new rows and positions."""
    h = 2
    c = Pair(wq, 2, h, 32, 11)
    k, v = _rows(4, h, "bf16", 3)
    s, o = _i32([0, 0]), _i32([0, 2, 4])
    wq.wq_kv_append(k, v, c.k, c.v, s, o)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ko = torch.empty(4, h, D, dtype=torch.bfloat16, device="cuda")
    vo = torch.empty_like(ko)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        wq.wq_kv_append(k, v, c.k, c.v, s, o)
        wq.wq_kv_read(c.k, c.v, s, o, 4, k_out=ko, v_out=vo)
    for cache, rows in zip(c.host, (k, v)):
        kvcache.append(cache, rows.float().cpu().numpy(), [0, 0], [0, 2, 4])
    for step, (starts, edges) in enumerate((([2, 5], [0, 1, 4]), ([9, 30], [0, 3, 4]))):
        nk, nv = _rows(4, h, "bf16", 40 + step)
        k.copy_(nk), v.copy_(nv), s.copy_(_i32(starts)), o.copy_(_i32(edges))
        graph.replay()
        for cache, rows, got in zip(c.host, (k, v), (ko, vo)):
            kvcache.append(cache, rows.float().cpu().numpy(), starts, edges)
            want = torch.from_numpy(kvcache.read(cache, starts, edges, 4)).to(torch.bfloat16)
            assert torch.equal(got.cpu(), want)
        c.check()

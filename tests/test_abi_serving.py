"""Refusals of the 4-bit serving entry points, on the host (no launch)."""

import ctypes

import pytest

A16, MIS = 0x10000, 0x10004


@pytest.fixture(scope="module")
def wq():
    from bit_weight_quantized_weights_b200 import build_lib
    build_lib.build()
    from bit_weight_quantized_weights_b200 import binding
    return binding


def _pair(a, b):
    return (ctypes.c_int64 * 2)(a, b)


def _append(wq, k=A16, v=A16, dt=0, t=4, h=2, d=128, ks=(256, 128), vs=(256, 128), b=2, starts=A16,
            offsets=A16, cap=16, c=(A16,) * 6):
    return wq.lib.wq_kv_append(k, v, dt, t, h, d, _pair(*ks), _pair(*vs), b, starts, offsets, cap,
                               *c, None)


def _read(wq, k=A16, v=A16, dt=0, t=4, h=2, d=128, ks=(256, 128), vs=(256, 128), b=2, starts=A16,
          offsets=A16, cap=16, c=(A16,) * 6):
    return wq.lib.wq_kv_read(*c, b, h, d, cap, starts, offsets, t, k, v, dt, _pair(*ks), _pair(*vs),
                             None)


@pytest.mark.parametrize("call", [_append, _read])
def test_kv_rows_validation(wq, call):
    assert call(wq, t=0) == wq.WQ_OK
    assert call(wq, b=0) == wq.WQ_OK
    for bad in (dict(t=-1), dict(h=0), dict(d=0), dict(b=-1), dict(cap=0), dict(dt=3), dict(k=None),
                dict(v=None), dict(starts=None), dict(offsets=None), dict(ks=(-256, 128)),
                dict(vs=(256, -128))):
        assert call(wq, **bad) == wq.WQ_ERR_INVALID_ARG, bad
    for i in range(6):
        c = [A16] * 6
        c[i] = None
        assert call(wq, c=c) == wq.WQ_ERR_INVALID_ARG
        c[i] = MIS
        assert call(wq, c=c) == wq.WQ_ERR_ALIGNMENT
    for bad in (dict(k=MIS), dict(v=MIS), dict(ks=(260, 128)), dict(vs=(256, 132)),
                dict(dt=2, ks=(256, 130)), dict(starts=A16 + 2), dict(offsets=A16 + 1)):
        assert call(wq, **bad) == wq.WQ_ERR_ALIGNMENT, bad
    for bad in (dict(d=64), dict(t=2 ** 31), dict(cap=2 ** 31 - 1), dict(b=65536),
                dict(t=2 ** 31 - 1, h=9)):
        assert call(wq, **bad) == wq.WQ_ERR_UNSUPPORTED, bad


def _attn(wq, q=A16, dt=0, stride=1024, b=2, hq=8, hkv=2, d=128, p=24, pcap=24, pre=(A16,) * 6,
          cap=16, own=(A16,) * 6, ln=A16, out=A16, ws=A16, n=1 << 40):
    return wq.lib.wq_prefix_attention(q, dt, stride, b, hq, hkv, d, p, pcap, *pre, cap, *own, ln,
                                      out, ws, n, None)


def test_prefix_attention_validation(wq):
    assert _attn(wq, b=0) == wq.WQ_OK
    for bad in (dict(b=-1), dict(hq=0), dict(hkv=0), dict(hq=9), dict(d=0), dict(p=-1), dict(cap=0),
                dict(p=25), dict(dt=2), dict(stride=-8), dict(q=None), dict(ln=None),
                dict(out=None), dict(pre=(None,) * 6), dict(own=(A16,) * 5 + (None,))):
        assert _attn(wq, **bad) == wq.WQ_ERR_INVALID_ARG, bad
    for bad in (dict(d=64), dict(hq=34), dict(cap=2 ** 31 - 1), dict(p=2 ** 31 - 1, pcap=2 ** 31),
                dict(pcap=2 ** 31 - 1), dict(cap=2 ** 30 + 1), dict(pcap=2 ** 30 + 1),
                dict(b=2 ** 28)):
        assert _attn(wq, **bad) == wq.WQ_ERR_UNSUPPORTED, bad
    for bad in (dict(q=MIS), dict(out=MIS), dict(ln=A16 + 2), dict(stride=1028), dict(ws=MIS),
                dict(pre=(A16, MIS) + (A16,) * 4), dict(own=(MIS,) + (A16,) * 5)):
        assert _attn(wq, **bad) == wq.WQ_ERR_ALIGNMENT, bad
    assert _attn(wq, ws=None) == wq.WQ_ERR_WORKSPACE
    size = ctypes.c_size_t()
    assert wq.lib.wq_prefix_attention_workspace(2, 8, 2, 128, 24, 16, ctypes.byref(size)) == wq.WQ_OK
    assert size.value > 0
    assert _attn(wq, n=size.value - 1) == wq.WQ_ERR_WORKSPACE
    assert wq.lib.wq_prefix_attention_workspace(0, 8, 2, 128, 24, 16,
                                                ctypes.byref(size)) == wq.WQ_OK
    assert size.value == 0
    assert wq.lib.wq_prefix_attention_workspace(2, 8, 2, 64, 24, 16,
                                                ctypes.byref(size)) == wq.WQ_ERR_UNSUPPORTED
    assert wq.lib.wq_prefix_attention_workspace(2, 8, 2, 128, 24, 16, None) == \
        wq.WQ_ERR_INVALID_ARG


def test_prefix_path_hook(wq):
    assert wq.lib.wq_test_set_prefix_path(3) == wq.WQ_ERR_INVALID_ARG
    assert wq.lib.wq_test_set_prefix_path(-1) == wq.WQ_ERR_INVALID_ARG
    sizes = []
    for path in (1, 2, 0):
        wq.wq_test_set_prefix_path(path)
        size = ctypes.c_size_t()
        assert wq.lib.wq_prefix_attention_workspace(64, 64, 8, 128, 32768, 1024,
                                                    ctypes.byref(size)) == wq.WQ_OK
        sizes.append(size.value)
    assert sizes[2] in sizes[:2] and min(sizes) > 0


def _planes(wq, x=A16, dt=0, ldx=512, m=4, k=512, n=2, c=A16, s=A16):
    return wq.lib.wq_mx_quantize_planes(x, dt, ldx, m, k, n, c, s, None)


def test_mx_planes_validation(wq):
    assert _planes(wq, m=0) == wq.WQ_OK
    for bad in (dict(m=-1), dict(k=0), dict(k=48), dict(ldx=504), dict(n=0), dict(n=3), dict(dt=3),
                dict(x=None), dict(c=None), dict(s=None)):
        assert _planes(wq, **bad) == wq.WQ_ERR_INVALID_ARG, bad
    for bad in (dict(x=MIS), dict(c=MIS), dict(s=MIS), dict(ldx=516), dict(dt=2, ldx=514)):
        assert _planes(wq, **bad) == wq.WQ_ERR_ALIGNMENT, bad
    for bad in (dict(m=2 ** 31), dict(m=2 ** 30, k=2048, ldx=2048)):
        assert _planes(wq, **bad) == wq.WQ_ERR_UNSUPPORTED, bad


def _gemm(wq, c=A16, s=A16, m=4, n=256, k=512, p=2, wc=A16, ws=A16, y=A16, w=A16, size=1 << 40):
    return wq.lib.wq_mx_gemm(c, s, m, n, k, p, wc, ws, y, w, size, None)


def test_mx_gemm_validation(wq):
    assert _gemm(wq, m=0) == wq.WQ_OK
    assert _gemm(wq, n=0) == wq.WQ_OK
    for bad in (dict(m=-1), dict(n=-1), dict(k=0), dict(k=48), dict(p=0), dict(p=3), dict(c=None),
                dict(s=None), dict(wc=None), dict(ws=None), dict(y=None)):
        assert _gemm(wq, **bad) == wq.WQ_ERR_INVALID_ARG, bad
    for bad in (dict(c=MIS), dict(s=MIS), dict(wc=MIS), dict(ws=MIS), dict(y=MIS), dict(w=MIS)):
        assert _gemm(wq, **bad) == wq.WQ_ERR_ALIGNMENT, bad
    for bad in (dict(k=96), dict(n=24), dict(m=2 ** 30), dict(n=2 ** 31), dict(k=2 ** 31),
                dict(m=2 ** 29, n=2 ** 20)):
        assert _gemm(wq, **bad) == wq.WQ_ERR_UNSUPPORTED, bad
    need = wq.wq_workspace_bytes(wq.WQ_OP_MX_GEMM, 4, 256, 512, 0, 2)
    assert need > 0
    assert _gemm(wq, w=None) == wq.WQ_ERR_WORKSPACE
    assert _gemm(wq, size=need - 1) == wq.WQ_ERR_WORKSPACE
    assert wq.wq_workspace_bytes(wq.WQ_OP_MX_GEMM, 0, 256, 512, 0, 2) == 0
    with pytest.raises(wq.WqError):
        wq.wq_workspace_bytes(wq.WQ_OP_MX_GEMM, 4, 256, 512, 0, 3)

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

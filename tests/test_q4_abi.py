"""4-bit entry points, checks that need no GPU: sizes of the packed form and the refusals
that the host makes before any CUDA call."""

import ctypes

import pytest

import dense_fp32_gemm_sgemm_gb300 as sg
from dense_fp32_gemm_sgemm_gb300 import build as sg_build

# fake, never dereferenced addresses
A, C, W_DATA, IDS, WEIGHTS, ROUTER = (0x10000000 * i for i in range(1, 7))
GATE, UP, DOWN = 0x700000000, 0x800000000, 0x900000000


class Q4(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("count", ctypes.c_int), ("N", ctypes.c_int),
                ("K", ctypes.c_int), ("group", ctypes.c_int), ("flags", ctypes.c_int)]


class Moe(ctypes.Structure):
    _fields_ = [("router", ctypes.c_void_p), ("router_dtype", ctypes.c_int),
                ("dtype", ctypes.c_int), ("D", ctypes.c_int), ("F", ctypes.c_int),
                ("E", ctypes.c_int), ("top_k", ctypes.c_int), ("renormalize", ctypes.c_int),
                ("gate", Q4), ("up", Q4), ("down", Q4)]


@pytest.fixture(scope="module")
def L():
    try:
        sg_build.nvcc()
    except RuntimeError:
        if not sg_build.up_to_date():
            pytest.skip("no nvcc and no prebuilt library")
    sg_build.build()
    return sg.lib()


def q4(data=W_DATA, count=1, N=256, K=64, group=64, flags=0):
    return Q4(data, count, N, K, group, flags)


@pytest.mark.parametrize("N,K,group,flags,count", [
    (128, 16, 128, 0, 1), (129, 17, 128, 0, 1), (1, 1, 32, 1, 1), (4096, 4096, 64, 3, 2),
    (65536, 1 << 20, 32, 1, 1)])
def test_packed_bytes(L, N, K, group, flags, count):
    unit = 8192 + 128 // group * 128 * (3 if flags & 1 else 2)
    want = count * -(-K // 128) * -(-N // 128) * unit
    assert L.sgemm_q4_bytes(ctypes.byref(q4(None, count, N, K, group, flags))) == want


BAD = [dict(count=0), dict(count=4097), dict(N=0), dict(N=65537), dict(K=0), dict(K=(1 << 20) + 1),
       dict(group=0), dict(group=16), dict(group=48), dict(group=256), dict(flags=4), dict(flags=-1)]


@pytest.mark.parametrize("bad", BAD, ids=lambda b: f"{list(b.items())[0]}")
def test_bad_descriptors_are_refused(L, bad):
    w = ctypes.byref(q4(**bad))
    assert L.sgemm_q4_bytes(w) == sg.ERR_ARG
    assert L.sgemm_q4_quantize(A, 0, 0, w, None) == sg.ERR_ARG
    assert L.sgemm_q4_pack(A, A, A, 0, w, None) == sg.ERR_ARG
    assert L.sgemm_q4_dequantize(w, A, None) == sg.ERR_ARG
    assert L.sgemm_q4_matmul(A, 0, 1 << 20, 1, w, C, 1 << 21, None) == sg.ERR_ARG


def test_null_and_misaligned_data_are_refused(L):
    assert L.sgemm_q4_bytes(None) == sg.ERR_ARG
    for w in (q4(data=None), q4(data=W_DATA + 8)):
        w = ctypes.byref(w)
        assert L.sgemm_q4_quantize(A, 0, 0, w, None) == sg.ERR_ARG
        assert L.sgemm_q4_pack(A, A, A, 0, w, None) == sg.ERR_ARG
        assert L.sgemm_q4_dequantize(w, A, None) == sg.ERR_ARG
        assert L.sgemm_q4_matmul(A, 0, 256, 1, w, C, 64, None) == sg.ERR_ARG
    w = ctypes.byref(q4())
    assert L.sgemm_q4_quantize(None, 0, 0, w, None) == sg.ERR_ARG
    assert L.sgemm_q4_pack(None, A, A, 0, w, None) == sg.ERR_ARG
    assert L.sgemm_q4_pack(A, None, A, 0, w, None) == sg.ERR_ARG
    assert L.sgemm_q4_pack(A, A, None, 0, ctypes.byref(q4(flags=1)), None) == sg.ERR_ARG
    assert L.sgemm_q4_dequantize(w, None, None) == sg.ERR_ARG
    assert L.sgemm_q4_matmul(None, 0, 256, 1, w, C, 64, None) == sg.ERR_ARG
    assert L.sgemm_q4_matmul(A, 0, 256, 1, w, None, 64, None) == sg.ERR_ARG


def test_bad_arguments_of_the_product_are_refused(L):
    w = ctypes.byref(q4())
    assert L.sgemm_q4_matmul(A, 3, 256, 1, w, C, 64, None) == sg.ERR_ARG
    assert L.sgemm_q4_matmul(A, -1, 256, 1, w, C, 64, None) == sg.ERR_ARG
    assert L.sgemm_q4_matmul(A, 0, 255, 1, w, C, 64, None) == sg.ERR_ARG
    assert L.sgemm_q4_matmul(A, 0, 256, 1, w, C, 63, None) == sg.ERR_ARG
    assert L.sgemm_q4_matmul(A, 0, 256, -1, w, C, 64, None) == sg.ERR_ARG
    assert L.sgemm_q4_matmul(A, 0, 256, 65537, w, C, 64, None) == sg.ERR_ARG
    assert L.sgemm_q4_matmul(A, 0, 256, 1, ctypes.byref(q4(count=2)), C, 64, None) == sg.ERR_ARG
    # no rows: nothing to do, whatever the pointers
    assert L.sgemm_q4_matmul(None, 0, 256, 0, w, None, 64, None) == sg.OK


def test_types_of_the_quantiser(L):
    assert L.sgemm_q4_quantize(A, 3, 0, ctypes.byref(q4()), None) == sg.ERR_ARG
    assert L.sgemm_q4_quantize(A, 0, 0, ctypes.byref(q4(flags=2)), None) == sg.ERR_UNSUPPORTED


def test_overlaps_are_refused(L):
    w = ctypes.byref(q4())
    size = L.sgemm_q4_bytes(w)
    for at in (W_DATA, W_DATA + size - 1, W_DATA - 3):
        assert L.sgemm_q4_quantize(at, 0, 0, w, None) == sg.ERR_OVERLAP
        assert L.sgemm_q4_pack(at, A, None, 0, w, None) == sg.ERR_OVERLAP
        assert L.sgemm_q4_pack(A, at, None, 0, w, None) == sg.ERR_OVERLAP
        assert L.sgemm_q4_dequantize(w, at, None) == sg.ERR_OVERLAP
        assert L.sgemm_q4_matmul(A, 0, 256, 1, w, at, 64, None) == sg.ERR_OVERLAP
    # the second of two rows of C reaches into A
    assert L.sgemm_q4_matmul(A, 0, 256, 2, w, A - 4 * 100, 100, None) == sg.ERR_OVERLAP


def moe(**kw):
    E, D, F = kw.get("E", 4), kw.get("D", 256), kw.get("F", 128)
    m = Moe(ROUTER, 0, 0, D, F, E, 2, 1, q4(GATE, E, D, F), q4(UP, E, D, F), q4(DOWN, E, F, D))
    for k, v in kw.items():
        setattr(m, k, v)
    return m


def call(L, m, x=A, ldx=256, T=2, live=None, y=C, ldy=256, ids=IDS, weights=WEIGHTS):
    return L.sgemm_moe(None if m is None else ctypes.byref(m), x, ldx, T, live, y, ldy, ids,
                       weights, None)


def test_bad_layers_are_refused(L):
    assert call(L, None) == sg.ERR_ARG
    for bad in (dict(router=None), dict(router_dtype=3), dict(dtype=-1), dict(D=0), dict(D=16385),
                dict(F=0), dict(F=16385), dict(E=0), dict(E=257), dict(top_k=0), dict(top_k=5),
                dict(E=32, top_k=17), dict(gate=q4(None, 4, 256, 128)),
                dict(gate=q4(GATE + 1, 4, 256, 128)), dict(up=q4(UP, 3, 256, 128)),
                dict(up=q4(UP, 4, 255, 128)), dict(up=q4(UP, 4, 256, 129)),
                dict(up=q4(UP, 4, 256, 128, 32)), dict(up=q4(UP, 4, 256, 128, 64, 1)),
                dict(down=q4(DOWN, 4, 256, 128)), dict(down=q4(DOWN, 4, 128, 256, 63))):
        m = moe(**bad)
        assert call(L, m, ldx=1 << 20, ldy=1 << 20) == sg.ERR_ARG, bad


def test_bad_arguments_of_the_layer_are_refused(L):
    m = moe()
    assert call(L, m, T=-1) == sg.ERR_ARG
    assert call(L, m, T=65) == sg.ERR_ARG
    assert call(L, m, ldx=255) == sg.ERR_ARG
    assert call(L, m, ldy=255) == sg.ERR_ARG
    assert call(L, m, x=None) == sg.ERR_ARG
    assert call(L, m, y=None) == sg.ERR_ARG
    assert call(L, m, x=None, y=None, T=0) == sg.OK


def test_overlaps_of_the_layer_are_refused(L):
    m = moe()
    assert call(L, m, y=A) == sg.ERR_OVERLAP
    assert call(L, m, y=ROUTER) == sg.ERR_OVERLAP
    assert call(L, m, y=DOWN + 16) == sg.ERR_OVERLAP
    assert call(L, m, ids=A + 64) == sg.ERR_OVERLAP
    assert call(L, m, weights=GATE) == sg.ERR_OVERLAP
    assert call(L, m, weights=IDS) == sg.ERR_OVERLAP
    assert call(L, m, ids=C) == sg.ERR_OVERLAP
    assert call(L, m, live=IDS + 1) == sg.ERR_OVERLAP

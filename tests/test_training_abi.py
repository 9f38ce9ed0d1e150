"""Training entry points, checks that need no GPU: the refusals that the host makes before any
CUDA call, and those of the binding."""

import ctypes

import pytest

import dense_fp32_gemm_sgemm_gb300 as sg
from dense_fp32_gemm_sgemm_gb300 import build as sg_build

torch = pytest.importorskip("torch")

# fake, never dereferenced addresses
X, W, Y, C, LOSS, LOSSES, LSE, DX, DW = (0x100000000 * i for i in range(1, 10))


class Ce(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("ldx", ctypes.c_longlong),
                ("weight", ctypes.c_void_p), ("ldw", ctypes.c_longlong),
                ("target", ctypes.c_void_p), ("target_bits", ctypes.c_int),
                ("dtype", ctypes.c_int), ("T", ctypes.c_int), ("D", ctypes.c_int),
                ("V", ctypes.c_int), ("token_weights", ctypes.c_void_p),
                ("loss", ctypes.c_void_p), ("losses", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("dx", ctypes.c_void_p), ("lddx", ctypes.c_longlong),
                ("dweight", ctypes.c_void_p), ("lddw", ctypes.c_longlong)]


@pytest.fixture(scope="module")
def L():
    try:
        sg_build.nvcc()
    except RuntimeError:
        if not sg_build.up_to_date():
            pytest.skip("no nvcc and no prebuilt library")
    sg_build.build()
    return sg.lib()


def ce(L, **kw):
    a = dict(x=X, ldx=64, weight=W, ldw=64, target=Y, target_bits=64, dtype=0, T=10, D=64, V=100,
             token_weights=C, loss=LOSS, losses=LOSSES, lse=LSE, dx=DX, lddx=64, dweight=DW, lddw=64)
    a.update(kw)
    return L.sgemm_cross_entropy(ctypes.byref(Ce(**a)), None)


@pytest.mark.parametrize("bad", [
    dict(dtype=-1), dict(dtype=3), dict(T=-1), dict(T=(1 << 20) + 1), dict(D=0), dict(D=65537),
    dict(V=0), dict(V=(1 << 20) + 1), dict(target_bits=16), dict(target_bits=0), dict(x=None),
    dict(weight=None), dict(target=None), dict(losses=None), dict(lse=None), dict(ldx=63),
    dict(ldw=63), dict(lddx=63), dict(lddw=63), dict(x=X + 2), dict(weight=W + 2),
    dict(target=Y + 4), dict(token_weights=C + 2), dict(loss=LOSS + 1), dict(losses=LOSSES + 2),
    dict(lse=LSE + 2), dict(dx=DX + 2), dict(dweight=DW + 1)], ids=lambda b: f"{list(b.items())[0]}")
def test_bad_arguments_of_the_loss_are_refused(L, bad):
    assert ce(L, **bad) == sg.ERR_ARG


def test_null_description_is_refused(L):
    assert L.sgemm_cross_entropy(None, None) == sg.ERR_ARG


@pytest.mark.parametrize("name,size", [("loss", 4), ("losses", 40), ("lse", 40), ("dx", 2560),
                                       ("dweight", 25600)])
def test_overlaps_of_the_loss_are_refused(L, name, size):
    for other, other_size in (("x", 2560), ("weight", 25600), ("target", 80), ("token_weights", 40)):
        at = dict(x=X, weight=W, target=Y, token_weights=C)[other]
        assert ce(L, **{name: at}) == sg.ERR_OVERLAP
        assert ce(L, **{name: at + other_size - 4}) == sg.ERR_OVERLAP
        assert ce(L, **{name: at - size + 4}) == sg.ERR_OVERLAP
    for other, at in (("losses", LOSSES), ("lse", LSE), ("dx", DX), ("dweight", DW)):
        if other != name:
            assert ce(L, **{name: at}) == sg.ERR_OVERLAP
    # the last row of a wide pitch counts
    assert ce(L, dx=W - 4 * 9 * 100, lddx=100) == sg.ERR_OVERLAP


COEF = (ctypes.c_float * 15)(*([3.4445, -4.775, 2.0315] * 5))


def ns(L, G=X, dtype=0, count=1, M=64, N=64, ldg=64, stride_g=4096, out=W, ldo=64, stride_o=4096,
       steps=5, coefficients=COEF, eps=1e-7):
    return L.sgemm_orthogonalize(G, dtype, count, M, N, ldg, stride_g, out, ldo, stride_o, steps,
                                 coefficients, eps, None)


@pytest.mark.parametrize("bad", [
    dict(dtype=3), dict(dtype=-1), dict(count=-1), dict(count=4097), dict(M=0), dict(N=0),
    dict(M=32769), dict(N=32769, ldg=40000, ldo=40000),
    dict(M=16385, N=16385, ldg=20000, ldo=20000), dict(ldg=63), dict(ldo=63), dict(steps=0),
    dict(steps=65), dict(coefficients=None), dict(eps=-1.0), dict(eps=float("nan")), dict(G=None),
    dict(out=None), dict(G=X + 2), dict(out=W + 1), dict(count=2, stride_g=4095),
    dict(count=2, stride_o=4095)], ids=lambda b: f"{list(b.items())[0]}")
def test_bad_arguments_of_the_update_are_refused(L, bad):
    assert ns(L, **bad) == sg.ERR_ARG


def test_overlaps_of_the_update_are_refused(L):
    assert ns(L, out=X + 4) == sg.ERR_OVERLAP
    assert ns(L, out=X, ldo=65) == sg.ERR_OVERLAP
    assert ns(L, out=X - 4 * 4095) == sg.ERR_OVERLAP
    assert ns(L, count=2, out=X, stride_o=5000) == sg.ERR_OVERLAP
    assert ns(L, count=0, G=None, out=None) == sg.OK  # nothing to do


def test_the_binding_refuses_what_is_not_on_a_gpu():
    x, w, y = torch.zeros(4, 8), torch.zeros(6, 8), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        sg.cross_entropy(x, w, y)
    with pytest.raises(TypeError, match="x must be a torch.Tensor"):
        sg.cross_entropy([1.0], w, y)
    with pytest.raises(ValueError, match="G must be a CUDA tensor"):
        sg.orthogonalize(x)
    with pytest.raises(ValueError, match="dx is given but not needed"):
        sg.cross_entropy_grad(x, w, y, need_dx=False, dx=x)

"""Values at the ends of FP32's range in the few-row product and the expert layer, with weights that
bring the results back into it.

Bounds as in test_q4_gpu.py and test_moe_gpu.py, with 2^-148 for results below FP32's normal range.
No sum that the definition has overflows in these tests.
"""

import pytest

import dense_fp32_gemm_sgemm_gb300 as sg
from tests.gpu_util import torch_cuda
from tests.test_moe_gpu import Case
from tests.test_q4_gpu import UNIT, dtypes, random_codes

pytestmark = pytest.mark.gpu

GROUPS = (32, 64, 128)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_fp32_gemm_sgemm_gb300 import build
    build.build()
    torch_cuda()


def matrix(key, count, N, K, group, zeros, factor):
    """A packed stack and its values; factor: by which each group's scales are multiplied."""
    torch = torch_cuda()
    codes, scales, z, _ = random_codes(key, count, N, K, group, zeros, False)
    f = torch.tensor(factor, dtype=torch.float64).view(1, -1, 1)
    scales = (scales.double() * f.cuda()).to(torch.bfloat16)  # some are subnormal
    at = torch.arange(N) // group
    base = z.cpu()[:, at].double() if zeros else 8.0
    values = (codes.cpu().double() - base) * scales.cpu().double()[:, at]
    return sg.q4_pack(codes, scales, z, group=group), values


def check(C, A, values, kind="f32"):
    ref, S = A.double() @ values, A.double().abs() @ values.abs()
    bound = 1e-5 * S + UNIT[kind] * ref.abs() + 2.0 ** -148
    err = (C.cpu().double() - ref).abs()
    assert (err <= bound).all(), f"{float((err / bound).max()):.3g} x the bound"


def one(*args):
    W, values = matrix(args[0], 1, *args[1:])
    return single(W), values[0]


def single(W):
    """A stack of one matrix as a matrix."""
    W.stack = False
    return W


@pytest.mark.parametrize("zeros", [False, True], ids=["sym", "zeros"])
@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("M", [1, 2, 11])
def test_f32_ends_of_the_range(M, group, zeros):
    """Rows near both ends of the range, by weights that bring the products back."""
    torch = torch_cuda()
    N, K = 256, 40
    gen = torch.Generator().manual_seed(M + group)
    for e, f in ((127, -30), (124, -110), (-120, 0), (-130, 40), (-138, 120), (100, -100)):
        W, values = one("ends", N, K, group, zeros, [2.0 ** f] * (N // group))
        sign = torch.where(torch.rand(M, N, generator=gen) < 0.5, -1.0, 1.0)
        A = ((torch.rand(M, N, generator=gen, dtype=torch.float64) + 0.9) * 2.0 ** e).float() * sign
        C = sg.q4_matmul(A.cuda(), W)
        assert torch.isfinite(C).all()
        check(C, A, values)


@pytest.mark.parametrize("M", [1, 9])
@pytest.mark.parametrize("group", GROUPS)
def test_f32_magnitudes_that_change_along_a_row(M, group):
    """Each group of n has a magnitude of its own, and scales that undo it."""
    torch = torch_cuda()
    N, K = 1024, 24
    G = N // group
    gen = torch.Generator().manual_seed(group)
    exponents = torch.randint(-140, 118, (G,), generator=gen)
    factor = [2.0 ** -max(-118, min(118, int(e))) for e in exponents]
    W, values = one("along", N, K, group, True, factor)
    A = torch.randn(M, N, generator=gen, dtype=torch.float64)
    A = (A * 2.0 ** exponents.double()[torch.arange(N) // group]).float()
    check(sg.q4_matmul(A.cuda(), W), A, values)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("M", [2, 11, 40])
def test_finite_special_values_beside_ordinary_rows(M, group, kind):
    """Values outside the plain form's range in some rows, at both ends of n."""
    torch = torch_cuda()
    N, K = 700, 50
    W, values = one("beside", N, K, group, True, [1.0] * -(-N // group))
    A = torch.randn(M, N, generator=torch.Generator().manual_seed(M + group)).to(dtypes()[kind])
    A[1, 3], A[1, N - 1] = 1e-25, 2.0 ** 26
    A[M - 1, 350] = -(2.0 ** 24)
    check(sg.q4_matmul(A.cuda(), W), A, values, kind)


def layer_case(T, kind, group, zeros, e_in, e_down, key):
    """A case whose gate and up scales are times 2^e_in, its down scales times 2^e_down; the routing
    does not depend on the tokens."""
    torch = torch_cuda()
    D, F, E = 130, 70, 2
    c = Case(T, D, F, E, 2, kind, group=group, zeros=zeros, key=key)
    mats, c.values = [], []
    for i, (n, k, e) in enumerate(((D, F, e_in), (D, F, e_in), (F, D, e_down))):
        W, values = matrix(("range", key, i), E, n, k, group, zeros, [2.0 ** e] * -(-n // group))
        mats.append(W)
        c.values.append(values)
    c.router.zero_()
    c.layer = sg.MoeLayer(c.router.cuda(), *mats, top_k=2, dtype=dtypes()[kind])
    return c


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("zeros", [False, True], ids=["sym", "zeros"])
@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("T", [1, 5, 20])
def test_layer_at_the_ends_of_the_range(T, group, zeros, kind):
    torch = torch_cuda()
    # tokens near an end of the range; then ordinary ones whose hidden values are near an end
    for x_exponent, e_in, e_down in ((122, -122, 0), (-122, 120, 0), (0, 57, -118), (0, -59, 110)):
        c = layer_case(T, kind, group, zeros, e_in, e_down, 95)
        x = (c.x.double() * 2.0 ** x_exponent).to(c.x.dtype)
        y, _, _ = c.check(x=x)
        assert torch.isfinite(y).all() and (y != 0).any()

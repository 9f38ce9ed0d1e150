"""float32 updates of few rows (or columns) against 64 bits: as near as the iteration in FP32, or 2^-20.

Near its end the iteration's products A A hold one large square in each sum of the diagonal; what the
accumulators cut off beside it must not show. FP32 arithmetic (a sum of n terms is off by some sqrt(n) 2^-24) ends
at 0.9 to 3e-6 here, and is taken as it is measured; 22 bits of X, A and the polynomial at 0.4 to 0.8e-6.
"""

import pytest

import dense_fp32_gemm_sgemm_gb300 as sg
from tests.gpu_util import torch_cuda
from tests.test_orthogonalize_gpu import A, B, C, iterate

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_fp32_gemm_sgemm_gb300 import build
    build.build()
    torch_cuda()


def in_fp32(g):
    x = g / (g.square().sum().sqrt() + 1e-7)
    for _ in range(5):
        gram = x @ x.mT
        x = A * x + (B * gram + C * (gram @ gram)) @ x
    return x


@pytest.mark.parametrize("kind", ["normal", "strong"])
@pytest.mark.parametrize("shape", [(42, 4851), (64, 999), (64, 8192), (71, 6384), (130, 1024), (512, 768),
                                   (600, 8000)], ids=str)
@pytest.mark.parametrize("tall", [False, True])
def test_as_near_as_fp32(shape, kind, tall):
    torch = torch_cuda()
    gen = torch.Generator(device="cuda").manual_seed(1)
    g = torch.randn(*shape, device="cuda", generator=gen)
    if kind == "strong":
        g += 4 * torch.randn(shape[0], 1, device="cuda", generator=gen) @ torch.randn(
            1, shape[1], device="cuda", generator=gen)
    want = iterate(g, ((A, B, C),) * 5)
    got = sg.orthogonalize(g.T.contiguous()).T if tall else sg.orthogonalize(g)
    err = float((got.double() - want).norm() / want.norm())
    plain = float((in_fp32(g).double() - want).norm() / want.norm())
    assert err <= 1.5 * plain + 2 ** -20, f"{err:.3g} against {plain:.3g} in FP32"
    assert sg.device_error() == sg.OK

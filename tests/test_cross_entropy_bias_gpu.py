"""Logits that are long sums of one sign: what the accumulators cut off, always towards zero, adds up and shows
in the mean of lse over the tokens.

Measured on sums of one sign, FP16 operands: an MMA loses up to two ulps of its accumulator (0.8 on average in
sums of 4 MMAs, 1.9 in sums of 32, 2.2 in the worst sum; bfloat16 products have fewer bits to lose: 0.3). An ulp
is 2^-23 of the accumulator at most, and as the sums grow evenly, the accumulator is half of a segment's sum on
average: n MMAs between two additions in FP32 lose at most n 2^-23 of their sum. n is 8 where tiles have 128
columns, 16 where the tokens are one row of tiles, 32 else. What rounds to nearest (additions of segments,
exponentials, lse itself) is 2^-22 of lse for a token at most, and averages out. So

    |mean(lse) - mean(lse in 64 bits)| <= (n 2^-23 + 2^-22) lse.
"""

import pytest

import dense_fp32_gemm_sgemm_gb300 as sg
from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_fp32_gemm_sgemm_gb300 import build
    build.build()
    torch_cuda()


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,V,n", [(1, 3000, 8), (256, 19000, 8), (1, 32768, 16), (200, 32768, 16),
                                   (256, 19457, 16), (300, 20000, 32)])
def test_long_positive_sums(T, V, n, name):
    torch = torch_cuda()
    dt = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]
    gen = torch.Generator(device="cuda").manual_seed(2)
    D = 2048
    x = (torch.rand(T, D, device="cuda", generator=gen) + 0.5).to(dt)
    w = ((torch.rand(V, D, device="cuda", generator=gen) + 0.5) / 64).to(dt)
    y = torch.randint(V, (T,), device="cuda", generator=gen)
    want = torch.logsumexp(x.double() @ w.double().T, -1)
    for out in (sg.cross_entropy(x, w, y), sg.cross_entropy_grad(x, w, y, need_dx=False)):
        off = float((out.lse.double() - want).mean() / want.mean())
        assert abs(off) <= n * 2 ** -23 + 2 ** -22, f"{off:.3g}"
    assert sg.device_error() == sg.OK

"""Updates whose products have long sums, of one sign: what the accumulators cut off adds up.

With the coefficients (0, 1, 0) a step is X' = A X, A = X X^T. All entries are positive, so that what an
accumulator loses at each MMA, always towards zero, shows in the result's projection onto the reference. That is
rounded as the result is: A's entries are nearly equal, and so are the results along a row or column of 64 to
192, so that their own roundings leave u / sqrt(3 * 20000) of a projection, 1.6e-5 for bfloat16. Nor do
bfloat16's factors of one FP16 piece average out: the entries have 193 different values, whose roundings to 11
bits leave 2^-11 / sqrt(3 * 193) = 2e-5 of a factor, three times over. So the reference is the product of the
rounded factors in 64 bits.

An MMA loses up to two ulps of its accumulator (measured: 1.9 on average in sums of 32 MMAs), an ulp is 2^-23
of it at most, and as the sums grow evenly the accumulator is half of a segment's sum on average: n MMAs between
two additions in FP32 lose at most n 2^-23 of their sum. n is 128 for 16-bit types, 36 for float32; the second
product's sum is one segment of 12 blocks of 16 at most: 12, or 36 in three products. Tolerance:
(n + 36) 2^-23, and 2^-18 for roundings that go the other way: a loss of 1.5e-5 turns 0.4 % of 20000 of them, by
2^-7, bfloat16, which is as much on average and off by 3e-6 / 2.
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


def first_piece(v, scale):
    return (v * scale).half().double() / scale


# 128 columns a tile; the stack has 256 with bfloat16
@pytest.mark.parametrize("shape", [(1, 64, 20000), (1, 20000, 64), (1, 100, 32000), (90, 192, 9000),
                                   (90, 9000, 192)], ids=str)
@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
def test_long_sums(shape, name):
    torch = torch_cuda()
    dt = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]
    gen = torch.Generator(device="cuda").manual_seed(1)
    g = (torch.rand(*shape, device="cuda", generator=gen) + 0.5).to(dt)
    got = sg.orthogonalize(g, steps=1, coefficients=(0.0, 1.0, 0.0))
    u = torch.finfo(dt).eps / 2
    for k, m in zip(got[:3], g[:3]):
        x = m.double()
        x = x / (x.norm() + 1e-7)
        want = (x @ x.mT) @ x if shape[1] <= shape[2] else x @ (x.mT @ x)
        ref = want
        if name == "bf16":
            f = first_piece(x, 2.0 ** 13)
            gram = first_piece(f @ f.mT if shape[1] <= shape[2] else f.mT @ f, 2.0 ** 12)
            ref = gram @ f if shape[1] <= shape[2] else f @ gram
        along = 1 + float(((k.double() - ref.to(dt).double()) * ref).sum() / ref.square().sum())
        n = 36 if name == "f32" else 128
        assert abs(along - 1) <= (n + 36) * 2 ** -23 + 2 ** -18, f"{along - 1:.3g}"
        # each element: the factors' roundings (A's, the polynomial's and X's) and its own
        each = (n + 36) * 2 ** -23 + u + (3 * 2 ** -11 if name == "bf16" else 2 ** -19)
        assert ((k.double() - want).abs() <= each * want).all()
    assert sg.device_error() == sg.OK

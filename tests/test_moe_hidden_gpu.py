"""Hidden values of the expert layer keep all 24 significant bits, whatever the layer's type.

Two hidden values that differ by a 4096th are subtracted by the second product, so that the
output is what their low bits hold. The weights are 0, 1 and -1 (zero points 0, one group for
each hidden value), so every product is exact and a hidden value's error is that of its own
FP32 arithmetic: both share silu(g), and each rounds once more when it is multiplied by u:
2^-24 of it. Its three pieces add up without loss but for the accumulator's last place (2^-22).
Bound: 2^-21 (|h0| + |h1|), 2^-20 |y| for silu, and half a unit of y's type.
"""

import pytest

import dense_fp32_gemm_sgemm_gb300 as sg
from tests.gpu_util import torch_cuda
from tests.test_q4_gpu import UNIT, dtypes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_fp32_gemm_sgemm_gb300 import build
    build.build()
    torch_cuda()


def sparse(N, K, ones, signs):
    """A stack of one N x K matrix: signs[g] at the places `ones` of group g of 32 rows."""
    torch = torch_cuda()
    codes = torch.zeros(1, N, K, dtype=torch.uint8)
    for n, k in ones:
        codes[0, n, k] = 1
    groups = -(-N // 32)
    scales = torch.tensor(signs, dtype=torch.bfloat16).view(1, groups, 1).repeat(1, 1, K)
    zeros = torch.zeros(1, groups, K, dtype=torch.uint8)
    return sg.q4_pack(codes.cuda(), scales.cuda(), zeros.cuda(), group=32)


@pytest.mark.parametrize("T", [1, 2, 3, 8, 64])
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_low_bits_of_hidden_values(kind, T):
    torch = torch_cuda()
    dtype = dtypes()[kind]
    D, F = 64, 64
    gate = sparse(D, F, [(0, 0), (0, 32)], [1.0, 1.0])
    up = sparse(D, F, [(0, 0), (0, 32), (32, 32)], [1.0, 1.0])
    down = sparse(F, D, [(n, k) for n in (0, 32) for k in range(D)], [1.0, -1.0])
    layer = sg.MoeLayer(torch.zeros(1, D, dtype=dtype, device="cuda"), gate, up, down, top_k=1)
    gen = torch.Generator().manual_seed(40 + T)
    for _ in range(8):
        a = torch.rand(T, generator=gen) + 0.5
        b = (torch.rand(T, generator=gen) + 0.5) * 2.0 ** -12
        x = torch.zeros(T, D, dtype=dtype)
        x[:, 0], x[:, 32] = a, b
        y = layer(x.cuda())[0].cpu().double()
        a, b = x[:, 0].double(), x[:, 32].double()
        silu = a * torch.sigmoid(a)
        want = (-silu * b).unsqueeze(1)
        bound = 2.0 ** -21 * (silu * (2 * a + b)).unsqueeze(1) + (2.0 ** -20 + UNIT[kind]) * want.abs()
        bound += 2.0 ** -25 if kind == "f16" else 0
        assert ((y - want).abs() <= bound).all()

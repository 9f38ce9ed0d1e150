"""Tokens whose weights are far apart: each keeps its own gradient, as far as the header says.

g is held over the largest weight, in float16 times 2^14: rounded twice, 2^-11 each (bfloat16 2^-8), or by half of
2^-38 where that is more. A token's dx, by its own norm, may so be off by the two roundings of each g (the logits,
below 16, by 2^-17 of the sums of their terms' sizes, add 2^-12 at most), the result's rounding, and 2^-39 over its
share of the largest weight, times the sizes of the weights' rows. At 2^-16 the last is 2^-23, and nothing; at
2^-24 it is 2^-15 of sums of 300 entries where dx is some 0.3 of them, one percent.
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
@pytest.mark.parametrize("share,off", [(2.0 ** -8, 0), (2.0 ** -16, 0), (2.0 ** -24, 0.01)])
def test_small_weights_beside_large_ones(share, off, name):
    torch = torch_cuda()
    dt = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]
    u = torch.finfo(dt).eps / 2
    gen = torch.Generator(device="cuda").manual_seed(50)
    T, D, V = 300, 128, 300
    x = torch.randn(T, D, device="cuda", generator=gen).to(dt)
    w = (torch.randn(V, D, device="cuda", generator=gen) / 8).to(dt)
    y = torch.randint(V, (T,), device="cuda", generator=gen)
    c = torch.full((T,), 2.0 ** 14, device="cuda")
    c[1::2] *= share
    dx = sg.cross_entropy_grad(x, w, y, token_weights=c, need_dweight=False).dx
    s = x.double() @ w.double().T
    g = torch.softmax(s, -1)
    g[torch.arange(T, device="cuda"), y] -= 1
    want = c[:, None].double() * (g @ w.double())
    err = (dx.double() - want)[1::2].norm(dim=-1) / want[1::2].norm(dim=-1)
    # |g| . |w| over the norm of dx: how far roundings of one sign could add up
    add = ((g.abs() @ w.double().abs()).norm(dim=-1) / (g @ w.double()).norm(dim=-1))[1::2]
    tol = add * (2 * u + 2 ** -12) + u + (off if name == "f16" else 0)
    assert (err <= tol).all(), f"{float(err.max()):.3g}"
    if name == "f16" and not off:
        assert float(err.max()) <= 8 * u  # as with equal weights, far below one percent

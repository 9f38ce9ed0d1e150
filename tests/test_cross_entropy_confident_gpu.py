"""The loss and its gradient where the target is far above the other classes.

The weights are the identity and x holds whole numbers, so the logits are x itself, exactly, and dx is g
itself: each of its sums has one product that is not zero. With e = exp(s - target's s) and
rest = sum of the others' e,

    loss = log1p(rest),   g[target] = -c rest / (1 + rest),   g[v] = c e[v] / (1 + rest).

Tolerances, relative: an exponential (argument's rounding, ex2) and the sum of 128 of them in a row, 64
additions of 2^-24, its joins with the other blocks' (an expf and an addition each, some ten): below 2^-16
together, for rest and so for the loss and the target's g. Rounding to the type: u = 2^-8, 2^-11, 2^-24; the
target's g once, the others' twice; c is a power of two, so that no more is rounded. But float16's steps are no
smaller than 2^-24: g is held times 2^14, so that half a step is 2^-39 of c, and of a result 2^-25 = 2^-37 c as
c = 2^12. (At a lead of 20 the others' g are below 2^-28.) A gradient of the weights sums g times x: the same
bounds times |x|, 2^-16 of the sum of magnitudes, and the result's rounding, which in float16 is infinite from
65504 on: 85 tokens with x = -3, g near one and c = 4096 reach 10^6.
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


# 64 and 128 columns a block
@pytest.mark.parametrize("T,V", [(40, 300), (1024, 5000)])
@pytest.mark.parametrize("lead", [20, 17, 14, 9, 1, 0, -3])
@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
def test_what_is_left_of_a_confident_token(name, lead, T, V):
    torch = torch_cuda()
    dt = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]
    u = torch.finfo(dt).eps / 2
    gen = torch.Generator(device="cuda").manual_seed(lead + 3)
    x = -torch.randint(3, (T, V), device="cuda", generator=gen).float()
    # first, middle and last columns of blocks, and of the last block
    ends = torch.tensor([0, 31, 63, 64, 65, 100, 127, 128, 191, 255, V - 2, V - 1], device="cuda")
    y = ends[torch.arange(T, device="cuda") % len(ends)]
    one = torch.arange(T, device="cuda")
    x[one, y] = float(lead)
    c = 4096.0
    w = torch.eye(V, device="cuda", dtype=dt)
    out = sg.cross_entropy_grad(x.to(dt), w, y, token_weights=torch.full((T,), c, device="cuda"))
    alone = sg.cross_entropy(x.to(dt), w, y)

    e = torch.exp(x.double() - lead)
    e[one, y] = 0
    rest = e.sum(-1)
    loss = torch.log1p(rest)
    for got in (out, alone):
        assert ((got.losses - loss).abs() <= 2 ** -16 * loss).all()
        assert ((got.lse - (loss + lead)).abs() <= 2 ** -16 * loss + 2 ** -24 * abs(lead + 1)).all()
    g = e / (1 + rest[:, None])
    tol = g * (2 * u + u * u + 2 ** -16) + (2 ** -39 + 2 ** -37 if name == "f16" else 0)
    g[one, y] = -rest / (1 + rest)
    tol[one, y] = -g[one, y] * (u + 2 ** -16)
    err = (out.dx.double() / c - g).abs()
    assert (err <= tol).all(), f"worst {float((err / tol).max()):.3g} of the bound"
    dw = g.T @ x.double()
    size = g.abs().T @ x.double().abs()
    bound = tol.T @ x.double().abs() + 2 ** -16 * size + u * dw.abs()
    got = out.dweight.double() / c
    near = (got - dw).abs() <= bound
    if name == "f16":
        near |= torch.isinf(got) & (got.sign() == dw.sign()) & ((dw.abs() + bound) * c >= 65504)
    assert near.all()
    assert sg.device_error() == sg.OK

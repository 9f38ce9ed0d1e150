"""Infinite logits of the target and of the others, each row by the definition: a target of -inf has an infinite
loss (and p = 0), a row of -inf alone has lse = -inf and no loss, +inf and NaN anywhere make a row's loss and lse NaN.
Rows beside them keep theirs: their sums take the same steps whatever the others hold."""

import pytest

import dense_fp32_gemm_sgemm_gb300 as sg
from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_fp32_gemm_sgemm_gb300 import build
    build.build()
    torch_cuda()


@pytest.mark.parametrize("name", ["bf16", "f16"])
@pytest.mark.parametrize("T,V", [(20, 300), (1024, 5000)])  # 64 and 128 columns a block
def test_rows_by_the_definition(name, T, V):
    torch = torch_cuda()
    dt = {"bf16": torch.bfloat16, "f16": torch.float16}[name]
    gen = torch.Generator(device="cuda").manual_seed(60)
    D, inf = 64, float("inf")
    x = torch.randn(T, D, device="cuda", generator=gen)
    x[:, :4] = 0
    w = torch.randn(V, D, device="cuda", generator=gen) / 8
    w[:, :4] = 0
    y = torch.randint(5, V, (T,), device="cuda", generator=gen)
    clean = sg.cross_entropy(x.to(dt), w.to(dt), y)
    # rows 1 to 4 of x have a one where w has its infinities
    x[1, 0] = x[2, 1] = x[3, 2] = x[4, 3] = 1.0
    w[y[1], 0] = -inf     # row 1: its target
    w[:, 1] = -inf        # row 2: everything
    w[(y[3] + 7) % V, 2] = inf  # row 3: another class
    w[y[4], 3] = inf      # row 4: its target
    # zero times infinity is NaN, so each of these rows gets a head with its own infinities alone
    for row, col in ((1, 0), (2, 1), (3, 2), (4, 3)):
        head = w.clone()
        head[:, [c for c in range(4) if c != col]] = 0
        out = sg.cross_entropy(x[row:row + 1].to(dt), head.to(dt), y[row:row + 1])
        loss, lse = float(out.losses[0]), float(out.lse[0])
        if row == 1:
            s = x[1].to(dt).double() @ head.to(dt).double().T
            assert loss == inf and abs(lse - float(torch.logsumexp(s, -1))) <= 2 ** -14
        elif row == 2:
            assert loss != loss and lse == -inf
        else:
            assert loss != loss and lse != lse
    # many rows at once, one of them NaN
    bad = x.clone()
    bad[:, :4] = 0
    bad[5, 9] = float("nan")
    out = sg.cross_entropy(bad.to(dt), torch.where(torch.isinf(w), 0, w).to(dt), y)
    others = torch.arange(T, device="cuda") != 5
    assert torch.isnan(out.losses[5]) and torch.isnan(out.lse[5])
    assert torch.equal(out.losses[others], clean.losses[others])
    assert torch.equal(out.lse[others], clean.lse[others])
    assert sg.device_error() == sg.OK


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
def test_a_single_class(name):
    """V = 1: no loss and no gradient, whatever the logit is."""
    torch = torch_cuda()
    dt = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]
    x = (torch.arange(70 * 3, device="cuda").reshape(70, 3) - 100).to(dt)
    w = torch.ones(1, 3, device="cuda", dtype=dt)
    out = sg.cross_entropy_grad(x, w, torch.zeros(70, dtype=torch.int64, device="cuda"))
    assert not out.losses.any() and not out.dx.any() and not out.dweight.any() and float(out.loss) == 0
    assert torch.equal(out.lse, x.float().sum(-1))

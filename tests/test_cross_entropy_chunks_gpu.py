"""The loss's gradients over several chunks of tokens where few of them count.

A chunk of 2^20 classes in 16 bits is 768 tokens. A call with 1500 tokens, of which at most 700 count, has its
counted tokens in the first chunk alone, and a second one with none: dweight then goes out as what the first
left in the sums (and zeros where no token counts at all). The same tokens passed alone are one chunk, of the
same tiles: the results are equal to the bit. A few tokens alone make smaller chunks, whose sums are taken in
another order.
"""

import pytest

import dense_fp32_gemm_sgemm_gb300 as sg
from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu

T, D, V = 1500, 24, 1 << 20


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_fp32_gemm_sgemm_gb300 import build
    build.build()
    torch_cuda()


def inputs(name):
    torch = torch_cuda()
    dt = {"bf16": torch.bfloat16, "f16": torch.float16}[name]
    gen = torch.Generator(device="cuda").manual_seed(40)
    w = (torch.randn(V, D, device="cuda", generator=gen) * D ** -0.5).to(dt)
    y = torch.randint(V, (T,), device="cuda", generator=gen)
    x = (torch.randn(T, D, device="cuda", generator=gen) + 8 * w[y].float()).to(dt)
    c = (torch.rand(T, device="cuda", generator=gen) + 0.25) * 4096
    return x, w, y, c


@pytest.mark.parametrize("name", ["bf16", "f16"])
def test_a_last_chunk_without_tokens(name):
    torch = torch_cuda()
    x, w, y, c = inputs(name)
    gen = torch.Generator(device="cuda").manual_seed(41)
    chosen = torch.randperm(T, device="cuda", generator=gen)[:700].sort().values
    masked = torch.full_like(y, -100)
    masked[chosen] = y[chosen]
    x[masked < 0] = float("nan")
    want = sg.cross_entropy_grad(x[chosen], w, y[chosen], token_weights=c[chosen])
    got = sg.cross_entropy_grad(x, w, masked, token_weights=c)
    assert torch.isfinite(want.dweight.float()).all() and want.dweight.any()
    assert torch.equal(got.dweight, want.dweight)
    assert torch.equal(got.loss, want.loss)
    for a, b in ((got.losses, want.losses), (got.lse, want.lse), (got.dx, want.dx)):
        assert torch.equal(a[chosen], b)
        assert not a[masked < 0].any()
    masked.fill_(-100)
    none = sg.cross_entropy_grad(x, w, masked, token_weights=c)
    assert not any(t.any() for t in none)
    assert sg.device_error() == sg.OK


@pytest.mark.parametrize("name", ["bf16", "f16"])
def test_the_first_few_count(name):
    torch = torch_cuda()
    x, w, y, c = inputs(name)
    want = sg.cross_entropy_grad(x[:5], w, y[:5], token_weights=c[:5])
    y[5:] = -100
    got = sg.cross_entropy_grad(x, w, y, token_weights=c)
    assert torch.equal(got.losses[:5], want.losses) and not got.losses[5:].any()
    u = torch.finfo(x.dtype).eps / 2
    # the same g; sums of 5 tokens' terms, and of 2^20 classes' in parts: 128 MMAs of 2^-23 a segment
    size = c[:5].double().sum() * x[:5].double().abs().amax()
    assert ((got.dweight - want.dweight).double().abs()
            <= 2 * u * want.dweight.double().abs() + 2 ** -16 * size * 2 ** -20).all()
    dx_size = 2 * c[:5, None].double() * w.double().abs().amax()
    assert ((got.dx[:5] - want.dx).double().abs()
            <= 2 * u * want.dx.double().abs() + 2 ** -16 * dx_size).all()
    assert not got.dx[5:].any()


def test_float16_in_two_chunks():
    """float16 sums over two chunks with live tokens, each token with its own weight, against 64 bits for the
    classes that are targets (g rounded twice, 2^-11, the target's once; held over the largest c times 2^14, so
    2^-39 of it absolute; logits, lse and accumulation as in test_cross_entropy_gpu.py)."""
    torch = torch_cuda()
    x, w, y, c = inputs("f16")
    y[:40] = torch.arange(40, device="cuda") % 8
    y[-40:] = torch.arange(40, device="cuda") % 8
    out = sg.cross_entropy_grad(x, w, y, token_weights=c)
    again = sg.cross_entropy_grad(x, w, y, token_weights=c)
    assert all(torch.equal(a, b) for a, b in zip(out, again))
    u = 2.0 ** -11
    classes = torch.cat([torch.arange(8, device="cuda"), y[40:140], y[-140:-40],
                         torch.tensor([V - 1], device="cuda")]).unique()
    dw = torch.zeros(len(classes), D, dtype=torch.float64, device="cuda")
    tol, size = torch.zeros_like(dw), torch.zeros_like(dw)
    for part in torch.arange(T, device="cuda").split(64):
        xs = x[part].double()
        s = xs @ w.double().T
        es = (xs.abs() @ w.double().abs().T).amax(-1) * 2 ** -17
        lse = torch.logsumexp(s, -1)
        el = es + 2 ** -16 + 2 ** -23 * lse.abs()
        assert ((out.lse[part] - lse).abs() <= el).all()
        p = torch.exp(s - lse[:, None])[:, classes]
        hit = y[part][:, None] == classes
        share = c[part, None].double()
        g = torch.where(hit, p - 1, p) * share
        dg = (p * (2 * u + es + el + 2 ** -20)[:, None] + hit * u * (1 - p)) * share \
            + 2.0 ** -38 * float(c.max())
        dw += g.T @ xs
        tol += dg.T @ xs.abs()
        size += g.abs().T @ xs.abs()
    tol += 2 ** -16 * size + u * dw.abs() + 2 ** -25
    err = (out.dweight[classes].double() - dw).abs()
    assert (err <= tol).all(), f"worst {float((err / tol).max()):.3g} of the bound"

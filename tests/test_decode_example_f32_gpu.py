"""The decoding example with float32 activations, whose logits can be held to 64 bits closely.

Each of some ten products and sums on the way is off by some 3e-7 of its result's norm (float32
sums of 256 terms); the norms carry that on without growth, and the residual sums add such errors
like independent terms: 1e-6 of the logits' spread as a standard deviation, 5e-6 for the largest of
some thousand. 2e-5 leaves a factor of four; a route that flips on a near tie is excluded, as a
token whose experts differ from the 64-bit model's.
"""

import pytest

import dense_fp32_gemm_sgemm_gb300 as sg
from tests.gpu_util import torch_cuda
from tests.test_decode_example_gpu import example  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def test_float32_logits_against_64_bits(example):  # noqa: F811
    torch = torch_cuda()
    model = example.Model(dtype=torch.float32)
    tokens = torch.arange(9, device="cuda") * 13
    got = model.logits(tokens).double()

    def normed(x):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)

    x = model.embedding[tokens].double()
    y = model.embedding[tokens]
    agree = torch.ones(9, dtype=torch.bool, device="cuda")
    for block in model.blocks:
        layer = block.experts
        gate, up, down = (sg.q4_dequantize(w).double() for w in (layer.gate, layer.up, layer.down))
        x = x + normed(x) @ sg.q4_dequantize(block.proj).double()
        y = y + sg.q4_matmul(example.normed(y), block.proj)
        part, ids, _ = layer(example.normed(y))
        y = y + part
        h = normed(x)
        p = torch.softmax(h @ layer.router.double().T, -1)
        top = p.topk(layer.top_k, -1).indices.sort(-1).values
        agree &= (top == ids).all(-1)
        share = torch.zeros_like(p).scatter(1, top, p.gather(1, top) / p.gather(1, top).sum(1, True))
        g, u = torch.einsum("td,edf->etf", h, gate), torch.einsum("td,edf->etf", h, up)
        x = x + torch.einsum("etf,efd,te->td", g * torch.sigmoid(g) * u, down, share)
    want = normed(x) @ sg.q4_dequantize(model.head).double()
    assert agree.any()
    assert ((got - want)[agree].abs() <= 2e-5 * want.std()).all()

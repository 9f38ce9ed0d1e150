"""The decoding example on the GPU: captured steps against single calls, and against 64 bits.

Single calls and replays run the same kernels on the same sizes, so tokens are the same. Against
64 bits: each of the bfloat16 model's roundings (normed rows, products, sums; 4 to a half block)
costs at most 2^-8 of what it rounds. With rows normed to one, logits of a unit-variance model and
two blocks, the errors of some 16 roundings add to the logits like independent terms of 2^-9 each:
4 * 2^-9 of their spread as a standard deviation, times 5 for the largest of some thousand, below
0.05 of the spread; routes that flip on a near tie are excluded by comparing tokens whose routes
agree (none but ties can differ).
"""

import importlib.util
import pathlib

import pytest

from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    from dense_fp32_gemm_sgemm_gb300 import build
    build.build()
    torch_cuda()
    path = pathlib.Path(__file__).parent.parent / "examples" / "decode_4bit.py"
    spec = importlib.util.spec_from_file_location("decode_4bit", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_replays_are_single_calls(example):
    torch = torch_cuda()
    model = example.Model()
    start = torch.tensor([3, 1, 4, 159, 26], device="cuda")
    replayed = example.Decoder(model, 5).run(start, 6)
    tokens = start
    for step in range(6):
        live = torch.ones(5, dtype=torch.bool, device="cuda")
        tokens = model.logits(tokens, live).float().argmax(-1)
        assert torch.equal(tokens, replayed[:, step])


def test_logits_against_64_bits(example):
    import dense_fp32_gemm_sgemm_gb300 as sg
    torch = torch_cuda()
    model = example.Model()
    tokens = torch.arange(7, device="cuda") * 11
    got = model.logits(tokens).double()

    def normed(x):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)

    x = model.embedding[tokens].double()
    agree = torch.ones(7, dtype=torch.bool, device="cuda")
    y = model.embedding[tokens]
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
        new = x.clone()
        for t in range(7):
            weight = p[t, top[t]] / p[t, top[t]].sum()
            for c, e in zip(weight, top[t]):
                g, u = h[t] @ gate[e], h[t] @ up[e]
                new[t] += c * ((g * torch.sigmoid(g) * u) @ down[e])
        x = new
    want = normed(x) @ sg.q4_dequantize(model.head).double()
    assert agree.any()
    assert ((got - want)[agree].abs() <= 0.05 * want.std()).all()


def test_dead_sequences_stay(example):
    torch = torch_cuda()
    decoder = example.Decoder(example.Model(), 3)
    decoder.live.copy_(torch.tensor([True, False, True]))
    out = decoder.run(torch.tensor([5, 6, 7], device="cuda"), 3)
    assert (out[1] == 6).all()

"""The training example on the GPU: its gradients against 64 bits, and a captured step against a
direct one.

The gradients are in float32: products of the FP32 mode (1e-5 of the sums of magnitudes), logits off
by that and by 2^-17 of theirs, sums of 512 tokens. Relative to a gradient's norm 1e-4 leaves room for
sums of magnitudes some ten times the sums."""

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
    path = pathlib.Path(__file__).parent.parent / "examples" / "train_step.py"
    spec = importlib.util.spec_from_file_location("train_step", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_gradients_against_64_bits(example):
    torch = torch_cuda()
    model = example.Model()
    tokens, target = example.batch(torch.Generator(device="cuda").manual_seed(1), 1000, 512)
    loss, dmatrix, dhead = model.gradients(tokens, target)
    m = model.matrix.double().requires_grad_()
    h = model.head.double().requires_grad_()
    s = (model.embedding[tokens].double() @ m) @ h.T
    want = torch.nn.functional.cross_entropy(s, target)
    want.backward()
    want = float(want.detach())
    assert abs(float(loss) - want) <= 1e-5 * want
    for got, g in ((dmatrix, m.grad), (dhead, h.grad)):
        assert (got.double() - g).norm() <= 1e-4 * g.norm()


def test_a_captured_step_is_a_direct_one(example):
    torch = torch_cuda()
    gen = torch.Generator(device="cuda").manual_seed(2)
    batches = [example.batch(gen, 1000, 512) for _ in range(3)]
    direct, captured = example.Model(), example.Model()
    tokens, target = (t.clone() for t in batches[0])
    example.Model(seed=3).step(tokens, target)  # loads the kernels
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = captured.step(tokens, target)
    for b in batches:
        want = direct.step(*b)
        tokens.copy_(b[0])
        target.copy_(b[1])
        graph.replay()
        assert torch.equal(loss, want)
    assert torch.equal(direct.matrix, captured.matrix)
    assert torch.equal(direct.head, captured.head)
    assert torch.isfinite(direct.matrix).all()

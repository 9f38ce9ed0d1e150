"""4-bit calls on a stream of their own: results never lie in memory that work pending on the
caller's current stream still uses, and are not reused while that stream reads them."""

import pytest

import dense_fp32_gemm_sgemm_gb300 as sg
from tests.gpu_util import torch_cuda
from tests.test_moe_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_fp32_gemm_sgemm_gb300 import build
    build.build()
    torch_cuda()


def late_writes(*tensors):
    """Blocks like the tensors, freed while the current stream still has writes to them ahead."""
    torch = torch_cuda()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    blocks = [torch.empty_like(t) for t in tensors]
    for b in blocks:
        b.view(-1).view(torch.uint8).fill_(0)  # loads the kernel, which may wait for the device
    torch.cuda._sleep(50_000_000)  # some tens of milliseconds
    for b in blocks:
        b.view(-1).view(torch.uint8).fill_(0xff)


def calls():
    torch = torch_cuda()
    gen = torch.Generator().manual_seed(90)
    B = torch.randn(640, 4096, generator=gen).cuda()
    A = torch.randn(4, 640, generator=gen).cuda()
    W = sg.q4_quantize(B)
    codes = torch.randint(0, 16, (640, 4096), generator=gen, dtype=torch.uint8).cuda()
    scales = torch.rand(5, 4096, generator=gen).to(torch.bfloat16).cuda()
    c = Case(6, 512, 128, 4, 2, "f32", key=91)
    x = c.x.cuda()
    return {
        "quantize": lambda s: [sg.q4_quantize(B, stream=s).data],
        "pack": lambda s: [sg.q4_pack(codes, scales, stream=s).data],
        "dequantize": lambda s: [sg.q4_dequantize(W, stream=s)],
        "matmul": lambda s: [sg.q4_matmul(A, W, stream=s)],
        "layer": lambda s: list(c.layer(x, stream=s)),
    }


@pytest.mark.parametrize("name", ["quantize", "pack", "dequantize", "matmul", "layer"])
def test_results_are_not_in_memory_still_written(name):
    torch = torch_cuda()
    call = calls()[name]
    want = [t.clone() for t in call(None)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    late_writes(*want)
    got = call(s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", ["quantize", "pack", "dequantize", "matmul", "layer"])
def test_results_stay_while_the_current_stream_reads_them(name):
    torch = torch_cuda()
    call = calls()[name]
    want = [t.clone() for t in call(None)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = call(s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(50_000_000)
    copies = [t.clone() for t in got]
    del got
    with torch.cuda.stream(s):
        for t in want:
            torch.empty_like(t).view(-1).view(torch.uint8).fill_(0xff)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copies, want))


@pytest.mark.parametrize("name", ["quantize", "pack", "dequantize", "matmul", "layer"])
def test_in_a_graph_on_a_stream_given(name):
    torch = torch_cuda()
    call = calls()[name]
    want = [t.clone() for t in call(None)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call(torch.cuda.current_stream())
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))

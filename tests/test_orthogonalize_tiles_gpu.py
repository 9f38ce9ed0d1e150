"""Updates against 64 bits block by block: a block that is missing, in another's place or not mirrored shows
in its own norm, which a bound on the whole matrix would hide in weak parts.

Tolerance: for a block, the RMS bound of test_orthogonalize_gpu.py (the roundings by simulation, the
accumulators' cut, the result's rounding) relative to the larger of the block's and the matrix's RMS, times
four, as errors are spread over the blocks by the factors' roundings; and for a single element sixteen times
that bound relative to the matrix's RMS, or the rounding of the element itself.
"""

import pytest

import dense_fp32_gemm_sgemm_gb300 as sg
from tests.gpu_util import torch_cuda
from tests.test_orthogonalize_gpu import A, B, C, dtype_of, iterate, matrix

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_fp32_gemm_sgemm_gb300 import build
    build.build()
    torch_cuda()


def graded(shape, name, seed):
    """Rows and columns whose sizes fall by a thousand from the first to the last."""
    torch = torch_cuda()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    g = torch.randn(*shape, device="cuda", generator=gen)
    for d in (0, 1):
        size = [1, 1]
        size[d] = shape[d]
        g *= torch.logspace(0, -1.5, shape[d], device="cuda").reshape(size)
    return g.to(dtype_of(name))


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["normal", "strong", "low", "graded"])
@pytest.mark.parametrize("shape", [(300, 333), (700, 640), (640, 1100), (1100, 400)], ids=str)
def test_block_by_block(shape, kind, name):
    torch = torch_cuda()
    g = graded(shape, name, 5) if kind == "graded" else matrix(shape, name, seed=5, kind=kind)
    triples = ((A, B, C),) * 5
    got = sg.orthogonalize(g).double()
    want = iterate(g, triples)
    model = iterate(g, triples, rounded=1 if name == "bf16" else 2)
    n = -(-max(shape) // 16) * (1 if name == "bf16" else 3)
    if name == "f32":
        n = min(n, 36)
    norm = want.norm()
    u = torch.finfo(g.dtype).eps / 2
    tol = float(2 * (model - want).norm() / norm + 8 * n * 2 ** -23 + u)
    err = got - want
    rms = float(norm / want.numel() ** 0.5)

    def blocks(t):
        t = torch.nn.functional.pad(t, (0, -t.shape[1] % 64, 0, -t.shape[0] % 32))
        return t.unflatten(0, (-1, 32)).unflatten(2, (-1, 64)).norm(dim=(1, 3))

    full = blocks(torch.ones_like(want))  # the root of a block's size
    off = blocks(err) / (4 * tol * torch.maximum(blocks(want), rms * full))
    assert float(off.max()) <= 1, f"block {divmod(int(off.argmax()), off.shape[1])}: {float(off.max()):.3g}"
    each = err.abs() / torch.maximum(16 * tol * torch.full_like(want, rms), u * want.abs())
    assert float(each.max()) <= 1, f"{float(each.max()):.3g}"
    assert sg.device_error() == sg.OK

"""Updates with rows, columns or whole matrices of small entries, each row or column by its own norm.

X is kept in two FP16 pieces, of X times 2^13 and of what that leaves times 2^24; A (2^12 and 2^23) and the
polynomial (2^10 and 2^21) likewise, bfloat16's in the first piece alone. The tolerance is computed as in
test_orthogonalize_gpu.py, for the row instead of the matrix: twice what the iteration in 64 bits with exactly
those roundings is off by, 8 n 2^-23 for the accumulators' cut (n MMAs between additions in FP32: 12 for
float32, as here the smaller side is below 512; 128 for the 16-bit types) and the result's rounding u.
"""

import pytest

import dense_fp32_gemm_sgemm_gb300 as sg
from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu

A, B, C = 3.4445, -4.7750, 2.0315


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_fp32_gemm_sgemm_gb300 import build
    build.build()
    torch_cuda()


def pieces(v, n, scale):
    out, rest = [], v * scale
    for k in range(n):
        p = (rest * 2.0 ** (11 * k)).half().double() * 2.0 ** (-11 * k)
        out.append(p / scale)
        rest = rest - p
    return out


def iterate(g, eps, rounded=0, steps=5):
    """In 64 bits; with `rounded` (1 or 2 pieces of a factor) the stated roundings."""
    x = g.double()
    x = x / (x.square().sum().sqrt() + eps)

    def product(p, q):
        return p[0] @ q[0] if rounded == 1 else p[0] @ q[0] + p[0] @ q[1] + p[1] @ q[0]

    for _ in range(steps):
        if rounded:
            px = pieces(x, 2, 2.0 ** 13)
            pa = pieces(product(px, [p.mT for p in px]), rounded, 2.0 ** 12)
            pp = pieces(B * sum(pa) + C * product(pa, pa), rounded, 2.0 ** 10)
            x = A * sum(px) + product(pp, px)
        else:
            gram = x @ x.mT
            x = A * x + (B * gram + C * (gram @ gram)) @ x
    return x


def matrix(shape, seed):
    torch = torch_cuda()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, device="cuda", generator=gen)


def dtype_of(name):
    torch = torch_cuda()
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def check(got, g, eps, name, which):
    """Norms of the errors of the rows in `which` against those rows' norms. g is wide."""
    torch = torch_cuda()
    want = iterate(g, eps)
    model = iterate(g, eps, 1 if name == "bf16" else 2)
    n = 12 if name == "f32" else 128
    norm = want[which].norm(dim=-1)
    tol = 2 * (model - want)[which].norm(dim=-1) / norm + 8 * n * 2 ** -23 \
        + torch.finfo(g.dtype).eps / 2
    err = (got.double() - want)[which].norm(dim=-1) / norm
    assert (err <= tol).all(), f"{float(err.max()):.3g} against {float(tol.max()):.3g}"
    return float(err.max())


# float16's own range ends at 2^-24 of its 65504, so a row of it 1e-4 of the others has most of its bits
@pytest.mark.parametrize("name,small", [("f32", 1e-3), ("f32", 1e-5), ("f32", 1e-6), ("bf16", 1e-3),
                                        ("bf16", 1e-7), ("f16", 1e-4)])
@pytest.mark.parametrize("shape", [(256, 256), (200, 700), (130, 1024)], ids=str)
@pytest.mark.parametrize("tall", [False, True])
def test_small_rows(shape, name, small, tall):
    g = matrix(shape, 3)
    g[7] *= small
    g[shape[0] - 1] *= small
    if name == "f16":
        g *= 2.0 ** 10
    g = g.to(dtype_of(name))
    got = sg.orthogonalize(g.T.contiguous()).T if tall else sg.orthogonalize(g)
    err = check(got, g, 1e-7, name, [7, shape[0] - 1])
    if name == "f32":
        assert err <= 2e-5  # the roundings above add next to nothing at these sizes
    check(got, g, 1e-7, name, slice(None))
    assert sg.device_error() == sg.OK


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("norm", [1e-9, 1e-11, 1e-12])
def test_matrices_far_below_eps(name, norm):
    """X starts at |G| / eps, and stays a small multiple of it: its bits are what is tested."""
    g = matrix((256, 256), 4)
    g = (g * (norm / float(g.norm()))).to(dtype_of(name))
    err = check(sg.orthogonalize(g), g, 1e-7, name, slice(None))
    if name == "f32":
        assert err <= 2e-5

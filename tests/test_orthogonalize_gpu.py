"""Orthogonalised updates on the GPU against the iteration in 64 bits.

Tolerance. The stated arithmetic rounds X to two FP16 pieces and the factors to one (bfloat16) or two
pieces each, of values times 2^13, 2^12 and 2^10. What that costs depends on the matrix (small
singular values are multiplied by up to 3.4445^5 in five steps, with whatever rounding put there), so
it is computed: the iteration in 64 bits with exactly those roundings, against the one without. The
kernel may be off (2-norm of the difference over that of the result) by twice as much, plus what its
accumulators cut off: at most 2^-23 for each of the n MMAs of an accumulator, in each of a step's three
products, a step's error being at most multiplied by 3.4445 in each later one as the polynomial has no
steeper slope (n is the reduction over 16, times 3 for two pieces, but 36 at most for float32):
8 n 2^-23 for five steps, where later steps' own terms weigh most; plus the rounding of the result, u
(2^-8, 2^-11, 2^-24). A single element may be off by 16 times the RMS bound.
"""

import pytest

import dense_fp32_gemm_sgemm_gb300 as sg
from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu

NAMES = ("f32", "bf16", "f16")
A, B, C = 3.4445, -4.7750, 2.0315


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_fp32_gemm_sgemm_gb300 import build
    build.build()
    torch_cuda()


def dtype_of(name):
    torch = torch_cuda()
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def pieces(v, n, scale):
    torch = torch_cuda()
    out, rest = torch.zeros_like(v), v * scale
    for _ in range(n):
        p = rest.half().double()
        out, rest = out + p, rest - p
    return out / scale


def iterate(g, triples, eps=1e-7, rounded=0):
    """The iteration in 64 bits; with `rounded` (1 or 2 pieces of a factor) its roundings."""
    torch = torch_cuda()
    tall = g.shape[-2] > g.shape[-1]
    x = g.double().mT if tall else g.double()
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    for a, b, c in triples:
        if rounded:
            x = pieces(x, 2, 2.0 ** 13)
            f = pieces(x, rounded, 2.0 ** 13)
            gram = pieces(f @ f.mT, rounded, 2.0 ** 12)
            x = a * x + pieces(b * gram + c * (gram @ gram), rounded, 2.0 ** 10) @ f
        else:
            gram = x @ x.mT
            x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.mT if tall else x


def check(got, g, triples=((A, B, C),) * 5, eps=1e-7):
    torch = torch_cuda()
    f32 = g.dtype == torch.float32
    many = 1 if g.dtype == torch.bfloat16 else 2
    want = iterate(g, triples, eps)
    model = iterate(g, triples, eps, many)
    assert torch.isfinite(got.double()).all()
    n = -(-max(g.shape[-2:]) // 16) * (1 if many == 1 else 3)
    if f32:
        n = min(n, 36)
    for k, w, m in zip(*(t.reshape(-1, *g.shape[-2:]).double() for t in (got, want, model))):
        norm = w.norm()
        tol = (2 * (m - w).norm() / norm + 8 * n * 2 ** -23 + torch.finfo(g.dtype).eps / 2)
        err = (k - w).norm() / norm
        assert err <= tol, f"{float(err):.3g} against {float(tol):.3g}"
        rms = norm / w.numel() ** 0.5
        assert (k - w).abs().max() <= 16 * tol * torch.maximum(rms, w.abs().max())


def matrix(shape, name, seed=0, kind="normal"):
    torch = torch_cuda()
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, device="cuda", generator=gen)

    g = normal(*shape)
    if kind == "strong":  # a few strong directions
        r = max(1, min(shape[-2:]) // 32)
        g = g + 6 * normal(*shape[:-1], r) @ normal(*shape[:-2], r, shape[-1]) / r ** 0.5
    elif kind == "low":
        r = max(1, min(shape[-2:]) // 4)
        g = normal(*shape[:-1], r) @ normal(*shape[:-2], r, shape[-1])
    return (g * 1e-3).to(dtype_of(name))


# single elements, rows and columns; tiles' borders; wide and tall; 256 and 128 columns a tile;
# stacks, one whose phases overlap
SHAPES = [(1, 1), (1, 300), (300, 1), (2, 3), (64, 64), (65, 127), (127, 65), (128, 129), (256, 256),
          (257, 255), (300, 1000), (1000, 300), (520, 513), (3, 40, 70), (5, 260, 130),
          (20, 192, 320), (9, 600, 256)]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_against_64_bits(shape, name):
    g = matrix(shape, name, seed=sum(shape))
    for steps in (1, 5):
        check(sg.orthogonalize(g, steps=steps), g, ((A, B, C),) * steps)
    assert sg.device_error() == sg.OK


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("kind", ["strong", "low"])
@pytest.mark.parametrize("shape", [(384, 384), (200, 700), (2304, 2560)], ids=str)
def test_other_spectra(shape, kind, name):
    g = matrix(shape, name, seed=3, kind=kind)
    check(sg.orthogonalize(g), g)


@pytest.mark.parametrize("name", NAMES)
def test_coefficients_of_each_step(name):
    triples = ((4.0, -8.0, 5.0), (3.0, -4.0, 1.75), (2.0, -1.5, 0.5), (1.5, -0.5, 0.0))
    g = matrix((192, 260), name, seed=4)
    check(sg.orthogonalize(g, steps=4, coefficients=triples), g, triples)
    assert len(sg.ORTHOGONALIZE_COEFFICIENTS) == 3


def test_singular_values_end_near_one():
    torch = torch_cuda()
    g = matrix((512, 768), "f32", seed=5)
    s = torch.linalg.svdvals(sg.orthogonalize(g).double())
    assert 0.6 < s.min() and s.max() < 1.25


@pytest.mark.parametrize("name", NAMES)
def test_a_power_of_two_does_not_matter(name):
    """With eps = 0, bit for bit: the norm takes any range of the type."""
    torch = torch_cuda()
    g = matrix((130, 200), "f16", seed=6, kind="strong").to(dtype_of(name))
    want = sg.orthogonalize(g, eps=0.0)
    scales = (2.0 ** 5, 2.0 ** -4) if name == "f16" else (2.0 ** 100, 2.0 ** -90, 2.0 ** 60)
    for f in scales:
        if torch.equal(g * f / f, g):  # not so where float16 entries fall below 2^-14 and lose bits
            assert torch.equal(sg.orthogonalize(g * f, eps=0.0), want)
    assert torch.equal(g * scales[0] / scales[0], g)


@pytest.mark.parametrize("name", NAMES)
def test_strides_in_place_and_zeros(name):
    torch = torch_cuda()
    g = matrix((3, 90, 77), name, seed=7)
    want = sg.orthogonalize(g)
    wide = torch.full((3, 95, 83), 5.0, device="cuda", dtype=g.dtype)
    part = wide[:, 2:92, 1:78]
    part.copy_(g)
    out = torch.full((3, 90, 100), 5.0, device="cuda", dtype=g.dtype)
    assert torch.equal(sg.orthogonalize(part, out=out[:, :, 8:85]), want)
    assert torch.equal(out[:, :, 8:85], want)
    assert (out[:, :, :8] == 5).all() and (out[:, :, 85:] == 5).all()
    assert torch.equal(sg.orthogonalize(part, out=part), want) and torch.equal(part, want)
    assert (wide[:, :2] == 5).all() and (wide[:, 92:] == 5).all() and (wide[:, :, 78:] == 5).all()
    # nothing and zeros; a zero row stays one
    assert sg.orthogonalize(g[:0]).shape == (0, 90, 77)
    assert not sg.orthogonalize(torch.zeros_like(g)).any()
    z = g[0].clone()
    z[5] = 0
    assert not sg.orthogonalize(z)[5].any()


@pytest.mark.parametrize("name", NAMES)
def test_a_matrix_with_a_nan_keeps_it_to_itself(name):
    torch = torch_cuda()
    g = matrix((4, 150, 100), name, seed=8)
    want = sg.orthogonalize(g)
    g[1, 3, 4] = float("nan")
    g[3, 0, 0] = float("inf")
    got = sg.orthogonalize(g)
    assert torch.isnan(got[1]).all() and torch.isnan(got[3]).all()
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])


@pytest.mark.parametrize("name", NAMES)
def test_graphs_and_streams(name):
    torch = torch_cuda()
    gs = [matrix(s, name, seed=9) for s in ((300, 500), (6, 140, 140))]
    want = [sg.orthogonalize(g) for g in gs]
    streams = [torch.cuda.Stream() for _ in gs]
    torch.cuda.synchronize()
    got = [[sg.orthogonalize(g, stream=s) for g, s in zip(gs, streams)] for _ in range(4)]
    torch.cuda.synchronize()
    for run in got:
        assert all(torch.equal(a, b) for a, b in zip(run, want))
    graphs, outs = [], []
    for g, s in zip(gs, streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs.append(sg.orthogonalize(g))
        graphs.append(graph)
    for g in gs:
        g.neg_()
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, -b) for a, b in zip(outs, want))
    assert sg.device_error() == sg.OK


def test_refusals_of_the_binding():
    torch = torch_cuda()
    g = matrix((20, 30), "bf16")
    for bad in (lambda: sg.orthogonalize(g.double()), lambda: sg.orthogonalize(g[0]),
                lambda: sg.orthogonalize(g.T), lambda: sg.orthogonalize(g, steps=0),
                lambda: sg.orthogonalize(g, coefficients=(1.0, 2.0)),
                lambda: sg.orthogonalize(g, steps=3, coefficients=((1, 2, 3),) * 2),
                lambda: sg.orthogonalize(g, out=torch.empty_like(g).float()),
                lambda: sg.orthogonalize(g, out=g.T), lambda: sg.orthogonalize(g[:, :0]),
                lambda: sg.orthogonalize(g[None].expand(3, -1, -1))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: sg.orthogonalize(g, eps=-1.0), lambda: sg.orthogonalize(g, steps=65),
                lambda: sg.orthogonalize(g[:10], out=g[1:11])):
        with pytest.raises(sg.SgemmError):
            bad()

"""The few-row product and the expert layer on every pattern of NaN, rows of a product beside other
rows, large values that meet zero weights, and reductions that are too long for the widest kernel.
Bounds as in test_q4_gpu.py.
"""

import pytest

import dense_fp32_gemm_sgemm_gb300 as sg
from tests.gpu_util import torch_cuda
from tests.test_moe_gpu import Case
from tests.test_q4_gpu import UNIT, dtypes, random_codes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_fp32_gemm_sgemm_gb300 import build
    build.build()
    torch_cuda()


def matrix(key, N, K, group, zeros):
    """A packed matrix and its values."""
    codes, scales, z, values = random_codes(key, 1, N, K, group, zeros, False)
    return sg.q4_pack(codes[0], scales[0], None if z is None else z[0], group=group), values[0]


def check(C, A, values, tol=1e-5, kind="f32"):
    ref, S = A.double() @ values, A.double().abs() @ values.abs()
    bound = tol * S + UNIT[kind] * ref.abs() + (2.0 ** -25 if kind == "f16" else 0)
    err = (C.cpu().double() - ref).abs()
    assert (err <= bound).all(), f"{float((err / bound).max()):.3g} x the bound"


@pytest.mark.parametrize("kind,bits", [("f32", [0x7f800001, 0x7f80ffff, -0x7fffff, 0x7fc00000]),
                                       ("bf16", [0x7f81, 0x7fff, -0x7f]),
                                       ("f16", [0x7c01, 0x7dff, -0x3ff])])
@pytest.mark.parametrize("M", [5, 40])
def test_any_nan_is_one(M, kind, bits):
    torch = torch_cuda()
    N, K = 200, 33
    W, values = matrix("nan", N, K, 64, False)
    A = torch.randn(M, N, generator=torch.Generator().manual_seed(M)).to(dtypes()[kind])
    raw = A.view(torch.int32 if kind == "f32" else torch.int16)
    for i, b in enumerate(bits):
        raw[i, 17 * i + 3] = b
    assert bool(torch.isnan(A[:len(bits)]).any(1).all())
    C = sg.q4_matmul(A.cuda(), W)
    assert bool(torch.isnan(C[:len(bits)]).all())
    clean = A[len(bits):]
    check(C[len(bits):], clean, values, kind=kind)


@pytest.mark.parametrize("kind,bits", [("f32", 0x7f800001), ("bf16", 0x7f81), ("f16", 0x7c01)])
@pytest.mark.parametrize("T", [3, 40])
def test_any_nan_is_one_in_the_layer(T, kind, bits):
    torch = torch_cuda()
    c = Case(T, 100, 48, 4, 2, kind, key=85)
    want, _, _ = c.check()
    x = c.x.clone()
    x.view(torch.int32 if kind == "f32" else torch.int16)[1, 9] = bits
    y, ids, _ = c.layer(x.cuda())
    assert ids[1].tolist() == [0, 1]
    assert bool(torch.isnan(y[1]).all())
    others = [t for t in range(T) if t != 1]
    assert torch.equal(y.cpu().double()[others], want[others])


@pytest.mark.parametrize("kind,rows", [("f32", 3), ("bf16", 12), ("f32", 9)])
def test_rows_do_not_depend_on_others(kind, rows):
    """A row has the same bits whatever ordinary values the others hold, and an infinity or NaN
    elsewhere leaves it within its bound."""
    torch = torch_cuda()
    N, K = 4096, 200
    W, values = matrix("rows", N, K, 64, True)
    gen = torch.Generator().manual_seed(rows)
    A = torch.randn(rows, N, generator=gen).to(dtypes()[kind])
    first = sg.q4_matmul(A.cuda(), W)
    other = torch.randn(rows, N, generator=gen).to(dtypes()[kind])
    other[1] = A[1]
    assert torch.equal(sg.q4_matmul(other.cuda(), W)[1], first[1])
    other[0, 5], other[rows - 1, 7] = float("inf"), float("nan")
    check(sg.q4_matmul(other.cuda(), W)[1:2], A[1:2], values, kind=kind)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("zeros", [False, True], ids=["sym", "zeros"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 13])
def test_large_values_that_meet_zero_weights(M, group, zeros, kind):
    """S leaves them out, but the products are aligned to them: 2^-10 of the group's scale times its
    largest |A| is added to the bound for each group, as the header states it."""
    torch = torch_cuda()
    N, K = 1000, 50
    codes, scales, z, values = random_codes("zero", 1, N, K, group, zeros, False)
    groups = -(-N // group)
    gen = torch.Generator().manual_seed(group + M)
    A = torch.randn(M, N, generator=gen)
    for g in range(groups):
        n = g * group + int(torch.randint(0, min(group, N - g * group), (1,), generator=gen))
        codes[0, n] = z[0, g] if zeros else 8
        values[0, n] = 0
        A[:, n] *= 2.0 ** 13
    A = A.to(dtypes()[kind])
    W = sg.q4_pack(codes[0], scales[0], None if z is None else z[0], group=group)
    ref, S = A.double() @ values[0], A.double().abs() @ values[0].abs()
    padded = torch.nn.functional.pad(A.double().abs(), (0, groups * group - N))
    largest = padded.view(M, groups, group).amax(-1)
    bound = 1e-5 * S + 2.0 ** -10 * (largest @ scales[0].double().abs().cpu())
    bound += UNIT[kind] * (ref.abs() + bound) + (2.0 ** -25 if kind == "f16" else 0)
    assert ((sg.q4_matmul(A.cuda(), W).cpu().double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("zeros", [False, True], ids=["sym", "zeros"])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("N", [20000, 40961, 65536])
@pytest.mark.parametrize("kind,M", [("f32", 5), ("bf16", 17), ("f16", 9)])
def test_long_reductions(kind, M, N, group, zeros):
    """Reductions whose columns fit only 16 or 8 at a time. Up to 65536 n, a warpgroup of a
    cluster of 8 adds the sums of 32 units of up to 4 groups one after another: 128 of 2^-24
    each instead of 64, so 2e-5 S covers all."""
    torch = torch_cuda()
    K = 130
    W, values = matrix("long", N, K, group, zeros)
    A = torch.randn(M, N, generator=torch.Generator().manual_seed(N + M)).to(dtypes()[kind])
    check(sg.q4_matmul(A.cuda(), W), A, values, tol=2e-5, kind=kind)
    A[2, N - 1] = float("inf")
    C = sg.q4_matmul(A.cuda(), W)
    keep = [i for i in range(M) if i != 2]
    check(C[keep], A[keep], values, tol=2e-5, kind=kind)
    assert not bool(torch.isfinite(C[2]).any())

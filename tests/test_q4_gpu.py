"""4-bit weights on the GPU: quantisation against the formulas in FP32 (bit for bit), packing
and dequantisation (bit for bit), and the few-row product against the definition in 64 bits.

Tolerance of the product, elementwise, for N <= 8192: 1e-5 S + u |C|, S = |A| . |B|. The
weights and the pieces of A are exact, so what is left is summation in FP32: in a group at
most 8 matrix instructions that each may lose 2^-22 of the terms' magnitudes (1.9e-6 S),
then at most 256 group sums in all with 2^-24 each, of which no more than 64 follow one
another in a warp (3.8e-6 S), then warps and pieces, at most 48 sums (2.9e-6 S); u is half
a unit in the last place of C's type: 2^-24, 2^-8 (bfloat16), 2^-11 (float16, and 2^-25
absolute below its normal range).
"""

import zlib

import numpy as np
import pytest

import dense_fp32_gemm_sgemm_gb300 as sg
from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu

GROUPS = (32, 64, 128)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_fp32_gemm_sgemm_gb300 import build
    build.build()
    torch_cuda()


def dtypes():
    torch = torch_cuda()
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def rng(*key):
    return np.random.default_rng(list(key))


def bf16(x):
    """float32 values rounded to bfloat16 (nearest even), as float32."""
    b = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7fff + ((b >> 16) & 1)) & 0xffff0000
    return b.astype(np.uint32).view(np.float32)


def quantize_ref(B, group, zeros):
    """The header's formulas in FP32, group by group; returns the values held."""
    N, K = B.shape
    out = np.zeros((N, K), np.float32)
    for n in range(0, N, group):
        w = B[n:n + group]
        hi = np.maximum(w.max(0), np.float32(0))
        lo = np.minimum(w.min(0), np.float32(0))
        if zeros:
            s = bf16(hi / np.float32(15) - lo / np.float32(15))
        else:
            s = bf16(np.maximum(hi, -lo) / np.float32(7))
        safe = np.where(s > 0, s, np.float32(1))
        if zeros:
            z = np.clip(np.rint(-lo / safe), 0, 15)
            q = np.clip(np.rint(w / safe) + z, 0, 15) - z
        else:
            q = np.clip(np.rint(w / safe), -8, 7)
        out[n:n + group] = np.where(s > 0, s * q, np.float32(0))
    return out


@pytest.mark.parametrize("zeros", [False, True], ids=["sym", "zeros"])
@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("N,K", [(1, 1), (31, 3), (128, 64), (129, 65), (300, 70), (513, 33)])
def test_quantize_matches_the_formulas(N, K, group, zeros):
    torch = torch_cuda()
    B = rng(1, N, K, group).standard_normal((N, K)).astype(np.float32)
    B[:, 0] *= np.float32(1e-6)
    if K > 2:
        B[:, 1] = 0
        B[:, 2] = np.abs(B[:, 2])
    for transposed in (False, True):
        src = torch.from_numpy(np.ascontiguousarray(B.T if transposed else B)).cuda()
        got = sg.q4_dequantize(sg.q4_quantize(src, group=group, zeros=zeros, transposed=transposed))
        assert np.array_equal(got.cpu().numpy(), quantize_ref(B, group, zeros))


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_quantize_16_bit_sources(kind):
    torch = torch_cuda()
    src = torch.randn(200, 100, generator=torch.Generator().manual_seed(3)).to(dtypes()[kind])
    want = quantize_ref(src.float().numpy(), 64, True)
    got = sg.q4_dequantize(sg.q4_quantize(src.cuda(), group=64, zeros=True))
    assert np.array_equal(got.cpu().numpy(), want)


def test_quantize_extreme_magnitudes():
    torch = torch_cuda()
    B = rng(2).standard_normal((64, 5)).astype(np.float32)
    B[:, 1] *= np.float32(3e-39)   # subnormal
    B[:, 2] *= np.float32(5e37)
    B[:, 3] = np.float32(3.4028235e38) * np.sign(B[:, 3])
    B[:, 4] = np.float32(1e-45)
    for zeros in (False, True):
        got = sg.q4_dequantize(sg.q4_quantize(torch.from_numpy(B).cuda(), group=32, zeros=zeros))
        want = quantize_ref(B, 32, zeros)
        assert np.isfinite(want).all()
        assert np.array_equal(got.cpu().numpy(), want)


def random_codes(key, count, N, K, group, zeros, f16):
    """codes, scales, zero points (torch, CUDA) and their values in 64 bits."""
    torch = torch_cuda()
    g = torch.Generator().manual_seed(zlib.crc32(repr((key, count, N, K, group, zeros, f16)).encode()))
    G = -(-N // group)
    codes = torch.randint(0, 16, (count, N, K), generator=g, dtype=torch.uint8)
    scales = (torch.rand(count, G, K, generator=g) * 0.1 + 1e-3) * \
        torch.where(torch.rand(count, G, K, generator=g) < 0.2, -1.0, 1.0)
    scales = scales.to(torch.float16 if f16 else torch.bfloat16)
    z = torch.randint(0, 16, (count, G, K), generator=g, dtype=torch.uint8) if zeros else None
    at = torch.arange(N) // group
    base = z[:, at].double() if zeros else 8.0
    values = (codes.double() - base) * scales.double()[:, at]
    return codes.cuda(), scales.cuda(), None if z is None else z.cuda(), values


@pytest.mark.parametrize("f16", [False, True], ids=["sbf16", "sf16"])
@pytest.mark.parametrize("zeros", [False, True], ids=["sym", "zeros"])
@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("count,N,K", [(1, 1, 1), (1, 127, 15), (1, 128, 16), (3, 130, 18),
                                       (2, 257, 129)])
def test_pack_and_dequantize(count, N, K, group, zeros, f16):
    codes, scales, z, values = random_codes("pack", count, N, K, group, zeros, f16)
    for transposed in (False, True):
        turn = (lambda t: t.transpose(-1, -2).contiguous()) if transposed else (lambda t: t)
        W = sg.q4_pack(turn(codes), turn(scales), None if z is None else turn(z), group=group,
                       transposed=transposed)
        assert W.shape == (count, N, K) and W.group == group
        assert np.array_equal(sg.q4_dequantize(W).cpu().numpy(), values.float().numpy())
    one = sg.q4_pack(codes[0].contiguous(), scales[0].contiguous(),
                     None if z is None else z[0].contiguous(), group=group)
    assert one.shape == (N, K)
    assert np.array_equal(sg.q4_dequantize(one).cpu().numpy(), values[0].float().numpy())


def test_pack_masks_codes_and_caps_zero_points():
    torch = torch_cuda()
    codes = torch.arange(256, dtype=torch.uint8).view(64, 4).cuda()
    scales = torch.ones(2, 4, dtype=torch.bfloat16, device="cuda")
    z = torch.full((2, 4), 200, dtype=torch.uint8, device="cuda")
    got = sg.q4_dequantize(sg.q4_pack(codes, scales, z, group=32))
    assert torch.equal(got, (codes & 15).float() - 15)


UNIT = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def assert_product(C, A, values, kind, what):
    ref = A.double() @ values
    S = A.double().abs() @ values.abs()
    bound = 1e-5 * S + UNIT[kind] * ref.abs() + (2.0 ** -25 if kind == "f16" else 0)
    err = (C.cpu().double() - ref).abs()
    assert (err <= bound).all(), f"{what}: {float((err / bound).max()):.3g} x the bound"


SHAPES = [(1, 1, 1), (1, 31, 16), (1, 128, 64), (2, 129, 17), (1, 512, 512), (3, 1000, 130),
          (5, 513, 257), (8, 300, 48), (9, 256, 96), (16, 384, 80), (17, 640, 31), (33, 128, 33),
          (64, 257, 64), (65, 130, 50), (200, 200, 40)]


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K, group, kind):
    torch = torch_cuda()
    zeros = (M + N) % 2 == 0
    codes, scales, z, values = random_codes("mm", 1, N, K, group, zeros, (N + K) % 2 == 0)
    W = sg.q4_pack(codes[0], scales[0], None if z is None else z[0], group=group)
    A = torch.randn(M, N, generator=torch.Generator().manual_seed(M * N + K)).to(dtypes()[kind])
    C = sg.q4_matmul(A.cuda(), W)
    assert C.dtype == A.dtype and C.shape == (M, K)
    assert_product(C, A, values[0], kind, f"{M}x{N}x{K}")


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(1, 8192, 1024), (4, 8191, 333), (1, 6144, 4096), (16, 4097, 2050),
                                   (40, 4096, 1000), (2, 256, 8191)])
def test_product_of_ordinary_sizes(M, N, K, kind):
    torch = torch_cuda()
    codes, scales, z, values = random_codes("big", 1, N, K, 128 if N % 2 else 64, True, False)
    W = sg.q4_pack(codes[0], scales[0], z[0], group=128 if N % 2 else 64)
    A = torch.randn(M, N, generator=torch.Generator().manual_seed(N + K)).to(dtypes()[kind])
    assert_product(sg.q4_matmul(A.cuda(), W), A, values[0], kind, f"{M}x{N}x{K}")


def simple_matrix(N, K, group=64, key="simple", zeros=False):
    codes, scales, z, values = random_codes(key, 1, N, K, group, zeros, False)
    return sg.q4_pack(codes[0], scales[0], None if z is None else z[0], group=group), values[0]


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("offset,pad", [(0, 8), (1, 0), (3, 5), (8, 1)])
@pytest.mark.parametrize("M", [3, 40])
def test_slices_and_unaligned_rows(M, offset, pad, kind):
    """A and C as slices of wider tensors at any offset; what lies around C stays."""
    torch = torch_cuda()
    N, K = 300, 70
    W, values = simple_matrix(N, K)
    gen = torch.Generator().manual_seed(offset * 10 + pad)
    wide = torch.randn(M, offset + N + pad, generator=gen).to(dtypes()[kind])
    out = torch.full((M, offset + K + pad), 7.0, dtype=dtypes()[kind], device="cuda")
    view = out[:, offset:offset + K]
    sg.q4_matmul(wide.cuda()[:, offset:offset + N], W, out=view)
    assert_product(view, wide[:, offset:offset + N], values, kind, "slice")
    out[:, offset:offset + K] = 7.0
    assert bool((out == 7.0).all())


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_infinities_and_nans_stay_in_their_row(kind):
    torch = torch_cuda()
    N, K, M = 200, 40, 11
    W, values = simple_matrix(N, K)
    A = torch.randn(M, N, generator=torch.Generator().manual_seed(5)).to(dtypes()[kind])
    A[2, 7], A[5, 199], A[9, 0] = float("inf"), float("nan"), float("-inf")
    C = sg.q4_matmul(A.cuda(), W).cpu().double()
    special = [2, 5, 9]
    clean = [i for i in range(M) if i not in special]
    assert_product(C[clean], A[clean], values, kind, "clean rows")
    ref = A.double() @ values
    for i in special:
        assert torch.equal(torch.isnan(C[i]), torch.isnan(ref[i]))
        fine = ~torch.isnan(ref[i])
        assert torch.equal(C[i][fine], ref[i][fine])


def test_f32_extremes_of_range():
    """Values near both ends of FP32's range are split into pieces without overflow."""
    torch = torch_cuda()
    W, values = simple_matrix(128, 32)
    for scale in (2.0 ** 110, 2.0 ** -100):
        A = torch.randn(2, 128, generator=torch.Generator().manual_seed(6)) * scale
        assert_product(sg.q4_matmul(A.cuda(), W), A, values, "f32", f"scale {scale}")


def test_results_are_reproducible_and_rows_independent():
    torch = torch_cuda()
    W, _ = simple_matrix(4096, 512)
    A = torch.randn(24, 4096, generator=torch.Generator().manual_seed(7)).cuda()
    first = sg.q4_matmul(A, W)
    for _ in range(3):
        assert torch.equal(sg.q4_matmul(A, W), first)


def test_no_rows():
    torch = torch_cuda()
    W, _ = simple_matrix(64, 32)
    C = sg.q4_matmul(torch.empty(0, 64, device="cuda"), W)
    assert C.shape == (0, 32)


def test_on_another_stream_and_in_a_graph():
    torch = torch_cuda()
    W, values = simple_matrix(1024, 256)
    A = torch.randn(4, 1024, generator=torch.Generator().manual_seed(8))
    dA = A.cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    C = sg.q4_matmul(dA, W, stream=s)
    s.synchronize()
    assert_product(C, A, values, "f32", "stream")
    out = torch.empty_like(C)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sg.q4_matmul(dA, W, out=out)
    dA.mul_(2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, C * 2)


def test_binding_refusals():
    torch = torch_cuda()
    W, _ = simple_matrix(64, 32)
    A = torch.zeros(2, 64, device="cuda")
    with pytest.raises(TypeError):
        sg.q4_matmul(A, torch.zeros(64, 32, device="cuda"))
    with pytest.raises(ValueError):
        sg.q4_matmul(A.cpu(), W)
    with pytest.raises(ValueError):
        sg.q4_matmul(A.double(), W)
    with pytest.raises(ValueError):
        sg.q4_matmul(A[:, :63], W)
    with pytest.raises(ValueError):
        sg.q4_matmul(torch.zeros(64, 2, device="cuda").T, W)
    with pytest.raises(ValueError):
        sg.q4_matmul(A[:1].expand(2, 64), W)
    with pytest.raises(ValueError):
        sg.q4_matmul(A, W, out=torch.zeros(2, 32, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        sg.q4_matmul(A, W, out=torch.zeros(3, 32, device="cuda"))
    with pytest.raises(sg.SgemmError):
        sg.q4_matmul(A, W, out=A.view(-1)[:64].view(2, 32))  # C overlaps A
    with pytest.raises(sg.SgemmError):
        sg.q4_quantize(torch.zeros(64, 32, device="cuda"), group=48)
    with pytest.raises(ValueError):
        sg.q4_quantize(torch.zeros(64, 32, device="cuda").T)
    with pytest.raises(ValueError):
        sg.q4_quantize(torch.zeros(0, 32, device="cuda"))
    codes = torch.zeros(64, 32, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        sg.q4_pack(codes, torch.ones(1, 32, device="cuda"), group=64)
    with pytest.raises(ValueError):
        sg.q4_pack(codes, torch.ones(2, 32, dtype=torch.bfloat16, device="cuda"), group=64)
    with pytest.raises(ValueError):
        sg.q4_matmul(A, sg.q4_pack(codes[None].contiguous(),
                                   torch.ones(1, 1, 32, dtype=torch.bfloat16, device="cuda"),
                                   group=64))


def test_large_matrix_offsets():
    """A packed matrix and a dequantised one past 2^31 elements: the last strips are right."""
    torch = torch_cuda()
    N, K = 32768, 139264  # 4.6e9 weights, 2.4 GB packed
    G = N // 128
    codes = torch.zeros(N, K, dtype=torch.uint8, device="cuda")
    tail = torch.randint(0, 16, (N, 48), dtype=torch.uint8, generator=torch.Generator().manual_seed(9))
    codes[:, K - 48:] = tail.cuda()
    scales = torch.full((G, K), 0.5, dtype=torch.bfloat16, device="cuda")
    W = sg.q4_pack(codes, scales, group=128)
    del codes, scales
    A = torch.randn(1, N, generator=torch.Generator().manual_seed(10))
    C = sg.q4_matmul(A.cuda(), W)[:, K - 48:].cpu().double()
    values = (tail.double() - 8) * 0.5
    ref, S = A.double() @ values, A.double().abs() @ values.abs()
    # four times as many chunks a warp as at N = 8192
    assert ((C - ref).abs() <= 4e-5 * S).all()
    B = sg.q4_dequantize(W)
    assert torch.equal(B[:, K - 48:].cpu().double(), values)
    assert bool((B[:, :K - 48] == -4.0).all())

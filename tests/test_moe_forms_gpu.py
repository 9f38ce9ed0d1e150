"""The expert layer where inputs or hidden values lie outside the range that the weights' plain
form takes ([2^-64, 2^24)): the values, and that a token's result has the same bits whatever the
other tokens of its experts hold. Bounds as in test_moe_gpu.py.
"""

import pytest

from tests.gpu_util import torch_cuda
from tests.test_moe_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_fp32_gemm_sgemm_gb300 import build
    build.build()
    torch_cuda()


def blind(case, *columns):
    """Takes columns of x out of the routing, so that values of any size there leave the logits
    as exactly known as the others do."""
    for j in columns:
        case.router[:, j] = 0
        case.layer.router[:, j] = 0
    return case


GROUPS = [(32, 32), (64, 64), (128, 128), (32, 128), (128, 64)]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("zeros", [False, True], ids=["sym", "zeros"])
@pytest.mark.parametrize("group,down_group", GROUPS)
def test_values_of_special_tokens(group, down_group, zeros, kind):
    """Tokens with a tiny and a large element among ordinary ones, all on the same experts."""
    torch = torch_cuda()
    c = blind(Case(9, 200, 96, 3, 3, kind, group=group, down_group=down_group, zeros=zeros, key=80),
              5, 131, 199)
    x = c.x.clone()
    want, _, _ = c.layer(x.cuda())
    x[1, 5] = 1e-25
    x[3, 131] = 2.0 ** 26
    x[4, 199], x[4, 5] = -3e7, 1e-30
    x[8] = 0
    x[8, 131] = 2.0 ** 25
    y, _, _ = c.check(x=x)
    keep = [0, 2, 5, 6, 7]
    assert torch.equal(y[keep], want.cpu().double()[keep])


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("zeros", [False, True], ids=["sym", "zeros"])
@pytest.mark.parametrize("group,down_group", GROUPS)
@pytest.mark.parametrize("T", [2, 5, 12])
def test_special_hidden_values_change_no_other_token(T, group, down_group, zeros, kind):
    """Ordinary inputs whose hidden values are below 2^-64, or 2^24 and above."""
    torch = torch_cuda()
    c = Case(T, 200, 96, 2, 2, kind, group=group, down_group=down_group, zeros=zeros, key=81)
    base, _, _ = c.check()
    others = [t for t in range(T) if t != 1]
    for factor in (2.0 ** -40, 2.0 ** 14):
        x = c.x.clone()
        x[1] *= factor
        if factor > 1:  # the logits grow too: routed by one column that stays as it was
            x[1, 0] = c.x[1, 0]
            router = c.router.clone()
            c.router[:, 1:] = 0
            c.layer.router[:, 1:] = 0
            base, _, _ = c.check()
            y, _, _ = c.check(x=x)
            c.router.copy_(router)
            c.layer.router.copy_(router)
        else:
            y, _, _ = c.check(x=x)
        assert torch.equal(y[others], base[others])
        base, _, _ = c.check()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_tiny_routing_weights_change_no_other_token(kind):
    """A token whose second expert has a weight of some 1e-20."""
    torch = torch_cuda()
    c = Case(7, 64, 48, 2, 2, kind, group=64, renorm=False, key=82)
    c.router.zero_()
    c.router[0, 0] = 1.0
    c.layer.router.copy_(c.router)
    c.x[:, 0] = 0
    base, _, _ = c.check()
    x = c.x.clone()
    x[4, 0] = 46.0
    y, _, weights = c.check(x=x)
    assert 0 < float(weights[4, 1]) < 2.0 ** -64
    others = [t for t in range(7) if t != 4]
    assert torch.equal(y[others], base[others])


def test_nan_and_infinity_in_hidden_values_stay_in_their_token():
    """Finite inputs whose hidden values overflow."""
    torch = torch_cuda()
    c = blind(Case(6, 130, 64, 2, 2, "f32", group=64, key=83), 7)
    base, _, _ = c.check()
    x = c.x.clone()
    x[2, 7] = 2.0 ** 90
    y, _, _ = c.layer(x.cuda())
    assert not torch.isfinite(y[2]).any()
    others = [0, 1, 3, 4, 5]
    assert torch.equal(y.cpu().double()[others], base[others])

"""The mixture-of-experts layer on the GPU against its definition in 64 bits.

Routing: the chosen experts' logits are at least those of the others, up to the error of a
FP32 sum (1e-5 of the terms' magnitudes), and their weights match to 1e-5 relative to one
(the error of a logit, at most 1e-5 times the sum of magnitudes, here below 100, in the
exponent: bound 2e-3 of the weight in the worst case; measured against the bound that
follows from the token's own sums). Output, elementwise, with the layer's own ids:
g and u carry 1e-5 of their sums of magnitudes (derived in test_q4_gpu.py); through
silu(g) u, whose slopes are at most 1.1 |u| and |silu(g)|, that gives dh; the hidden values
lose 2^-14 for 16-bit types (two pieces) and nothing for float32; the weights' error is
that of the routing; the product back adds 1e-5 of its sum of magnitudes, and the output
half a unit of its type.
"""

import numpy as np
import pytest

import dense_fp32_gemm_sgemm_gb300 as sg
from tests.gpu_util import torch_cuda
from tests.test_q4_gpu import UNIT, dtypes, random_codes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_fp32_gemm_sgemm_gb300 import build
    build.build()
    torch_cuda()


class Case:
    def __init__(self, T, D, F, E, top, kind, group=64, zeros=False, f16=False, renorm=True,
                 router_kind=None, key=0, down_group=None):
        torch = torch_cuda()
        g = torch.Generator().manual_seed(1000 + key)
        self.T, self.D, self.F, self.E, self.top, self.kind = T, D, F, E, top, kind
        self.renorm = renorm
        self.x = torch.randn(T, D, generator=g).to(dtypes()[kind])
        self.router = (torch.randn(E, D, generator=g) * D ** -0.5).to(dtypes()[router_kind or kind])
        self.values, mats = [], []
        for i, (n, k) in enumerate(((D, F), (D, F), (F, D))):
            codes, scales, z, values = random_codes(("moe", key, i), E, n, k,
                                                    (down_group or group) if i == 2 else group,
                                                    zeros, f16)
            # keep the outputs' size about that of the inputs
            factor = 2.0 ** np.round(np.log2(4.0 * n ** -0.5))
            mats.append(sg.q4_pack(codes, (scales.float() * factor).to(scales.dtype), z,
                                   group=(down_group or group) if i == 2 else group))
            self.values.append(values * factor if not f16 else
                               sg.q4_dequantize(mats[-1]).cpu().double())
        self.layer = sg.MoeLayer(self.router.cuda(), *mats, top_k=top, renormalize=renorm,
                                 dtype=dtypes()[kind])

    def check(self, live=None, x=None):
        torch = torch_cuda()
        x = self.x if x is None else x
        y, ids, weights = self.layer(x.cuda(), live=None if live is None else live.cuda())
        y, ids, weights = y.cpu().double(), ids.cpu(), weights.cpu().double()
        X, R = x.double(), self.router.double()
        logits, mags = X @ R.T, X.abs() @ R.abs().T
        gate, up, down = self.values
        for t in range(x.shape[0]):
            if live is not None and not bool(live[t]):
                assert (ids[t] == -1).all() and (weights[t] == 0).all() and (y[t] == 0).all()
                continue
            chosen = ids[t].tolist()
            assert chosen == sorted(set(chosen)) and 0 <= chosen[0] and chosen[-1] < self.E
            slack = 2e-5 * float(mags[t].max())
            rest = [e for e in range(self.E) if e not in chosen]
            if rest:
                assert min(logits[t][chosen]) >= max(logits[t][rest]) - slack
            p = torch.softmax(logits[t], 0)[chosen]
            c = p / p.sum() if self.renorm else p
            rel = 2 * slack + 1e-6
            assert ((weights[t] - c).abs() <= rel * c + 1e-30).all()
            ref, bound = torch.zeros(self.D).double(), torch.zeros(self.D).double()
            for w, e in zip(c.tolist(), chosen):
                g, u = X[t] @ gate[e], X[t] @ up[e]
                dg, du = (1e-5 * (X[t].abs() @ m[e].abs()) for m in (gate, up))
                s = g * torch.sigmoid(g)
                h = s * u
                dh = 1.1 * dg * u.abs() + (s.abs() + 1.1 * dg) * du + 1e-6 * h.abs()
                dh += (0 if self.kind == "f32" else 2.0 ** -14) * h.abs()
                dh += rel * h.abs()
                ref += w * (h @ down[e])
                bound += w * ((dh + 1e-5 * h.abs()) @ down[e].abs())
            bound += UNIT[self.kind] * (ref.abs() + bound) + (2.0 ** -25 if self.kind == "f16" else 0)
            err = (y[t] - ref).abs()
            assert (err <= bound).all(), f"token {t}: {float((err / bound).max()):.3g} x the bound"
        return y, ids, weights


CASES = [(1, 64, 32, 2, 1), (1, 512, 256, 8, 2), (2, 129, 17, 3, 3), (3, 1, 1, 4, 2),
         (5, 300, 130, 7, 3), (8, 256, 512, 16, 4), (17, 130, 70, 33, 5), (64, 192, 100, 12, 6),
         (33, 257, 65, 256, 16), (9, 640, 48, 1, 1)]


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_layer(case, kind):
    T, D, F, E, top = CASES[case]
    c = Case(T, D, F, E, top, kind, group=(32, 64, 128)[case % 3], zeros=case % 2 == 1,
             f16=case % 4 == 3, renorm=case % 3 != 1, key=case, down_group=(64, 32, 128)[case % 3])
    c.check()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_every_token_picks_the_same_experts(kind):
    """All tokens on the same experts: the most columns an expert can get."""
    torch = torch_cuda()
    c = Case(64, 200, 96, 16, 2, kind, key=50)
    x = c.x[:1].repeat(64, 1)
    y, ids, _ = c.check(x=x)
    assert (y == y[0]).all() and (ids == ids[0]).all()


def test_larger_layer():
    Case(4, 2048, 1024, 8, 2, "bf16", group=128, key=51).check()
    Case(2, 1024, 2050, 8, 2, "f32", group=128, key=52).check()


@pytest.mark.parametrize("alive", [[], [0], [2, 3, 6], list(range(7))])
def test_live_mask(alive):
    torch = torch_cuda()
    c = Case(7, 130, 48, 6, 2, "bf16", key=60)
    live = torch.zeros(7, dtype=torch.bool)
    live[alive] = True
    y, _, _ = c.check(live=live)
    c.check(live=live.to(torch.uint8) * 3)
    full, _, _ = c.check()
    assert torch.equal(y[alive], full[alive])  # a token's result does not depend on the others


def test_masked_tokens_may_hold_anything():
    torch = torch_cuda()
    c = Case(5, 200, 64, 6, 2, "f32", key=61)
    live = torch.tensor([True, False, True, False, True])
    want, _, _ = c.check(live=live)
    x = c.x.clone()
    x[1], x[3] = float("nan"), float("inf")
    y, ids, weights = c.layer(x.cuda(), live=live.cuda())
    assert torch.equal(y.cpu().double(), want)
    assert (ids[1] == -1).all() and (weights[3] == 0).all()


def test_nan_token_stays_alone():
    torch = torch_cuda()
    c = Case(4, 200, 64, 6, 3, "f32", key=62)
    want, want_ids, _ = c.check()
    x = c.x.clone()
    x[2, 5] = float("nan")
    y, ids, _ = c.layer(x.cuda())
    assert ids[2].tolist() == [0, 1, 2]  # all logits NaN: the lowest indices
    assert torch.isnan(y[2]).all()
    keep = [0, 1, 3]
    assert torch.equal(y.cpu().double()[keep], want[keep])
    assert torch.equal(ids.cpu()[keep], want_ids[keep])


def test_ties_go_to_the_lowest_index():
    torch = torch_cuda()
    E, D = 40, 64
    c = Case(3, D, 32, E, 4, "f32", key=63)
    c.layer.router.zero_()
    c.layer.router[7:] = 1.0   # experts 7.. tie above 0..6 for positive sums
    x = torch.ones(3, D)
    x[1] = -1.0                # then 0..6 tie above the others
    x[2] = 0.0                 # and here all tie
    _, ids, weights = c.layer(x.cuda())
    assert ids.tolist() == [[7, 8, 9, 10], [0, 1, 2, 3], [0, 1, 2, 3]]
    assert torch.equal(weights.cpu(), torch.full((3, 4), 0.25))


def test_large_logits_do_not_overflow():
    torch = torch_cuda()
    c = Case(2, 64, 32, 5, 2, "f32", key=64)
    c.layer.router.mul_(1e6)
    _, ids, weights = c.layer(c.x.cuda())
    assert torch.isfinite(weights).all() and (weights.sum(1) - 1).abs().max() < 1e-6


def test_no_tokens():
    torch = torch_cuda()
    c = Case(1, 64, 32, 4, 2, "bf16", key=65)
    y, ids, weights = c.layer(c.x.cuda()[:0])
    assert y.shape == (0, 64) and ids.shape == (0, 2) and weights.shape == (0, 2)


@pytest.mark.parametrize("offset,pad", [(1, 2), (8, 8)])
def test_slices(offset, pad):
    torch = torch_cuda()
    c = Case(6, 128, 64, 8, 2, "bf16", key=66)
    want, _, _ = c.check()
    wide = torch.zeros(6, offset + 128 + pad, dtype=torch.bfloat16, device="cuda")
    wide[:, offset:offset + 128] = c.x.cuda()
    out = torch.full((6, offset + 128 + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    c.layer(wide[:, offset:offset + 128], out=out[:, offset:offset + 128])
    assert torch.equal(out[:, offset:offset + 128].cpu().double(), want)
    out[:, offset:offset + 128] = 7.0
    assert bool((out == 7.0).all())


def test_reproducible_on_streams_and_in_graphs():
    torch = torch_cuda()
    c = Case(12, 512, 300, 16, 4, "bf16", key=67)
    x = c.x.cuda()
    first = c.layer(x)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(c.layer(x), first))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = c.layer(x, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, first))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = c.layer(x)
    for _ in range(3):
        out[0].fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, first))
    assert sg.device_error() == sg.OK


def test_calls_on_two_streams_at_once():
    torch = torch_cuda()
    c = Case(8, 1024, 512, 16, 2, "bf16", group=128, key=68)
    x = c.x.cuda()
    want = c.layer(x)[0]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    torch.cuda.synchronize()
    for _ in range(20):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(c.layer(x)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    assert sg.device_error() == sg.OK


def test_binding_refusals():
    torch = torch_cuda()
    c = Case(2, 64, 32, 4, 2, "bf16", key=69)
    L, x = c.layer, c.x.cuda()
    for bad in (x.float(), x.cpu(), x[:, :63], x[:1].expand(2, 64),
                torch.zeros(65, 64, dtype=torch.bfloat16, device="cuda")):
        with pytest.raises(ValueError):
            L(bad)
    with pytest.raises(ValueError):
        L(x, live=torch.ones(3, dtype=torch.bool, device="cuda"))
    with pytest.raises(ValueError):
        L(x, live=torch.ones(2, device="cuda"))
    with pytest.raises(ValueError):
        L(x, out=torch.empty(2, 64, device="cuda"))
    with pytest.raises(sg.SgemmError):
        L(x, out=x)
    for args, top in (((L.up, L.gate, L.gate), 2), ((L.gate, L.up, L.down), 5),
                      ((L.gate, L.up, L.down), 0), ((L.gate, L.down, L.down), 2)):
        with pytest.raises(ValueError):
            sg.MoeLayer(L.router, *args, top_k=top)
    with pytest.raises(TypeError):
        sg.MoeLayer(L.router, L.gate, L.up, L.router, top_k=2)

"""Cross entropy on the GPU against its definition in 64 bits.

Tolerances, with S[t][v] = |x[t]| . |w[v]| and u half a unit in the last place of the type (2^-8
bfloat16, 2^-11 float16, 2^-24 float32):

 * a logit: the accumulator may lose 2^-23 of itself in each of the 64 MMAs of a segment (32 for
   float32), the segments' sums are FP32, and float32's dropped pieces are below 2^-23 of a product:
   es = 2^-17 S (2^-18 * 1.5 S for float32);
 * lse: the largest es, the exponentials and their sums (FP32, a block of 128 in a row, then a tree:
   below 2^-16 of the sum), and the rounding of the result: el = max es + 2^-16 + 2^-23 |lse|; a loss
   twice that;
 * g[t][v], of p = exp(s - lse): two roundings to the type (three pieces for float32: 2^-23), the
   logit's and lse's errors and the exponential functions' (2^-20): p (2 u + es + el + 2^-20); the
   target's p - 1 is rounded once, u |p - 1|, and p in it is off by p (es + el + 2^-20). float16 keeps
   exponentials down to 2^-40 of a block's largest and g down to 2^-39 of the largest c; FP32 and
   bfloat16 end at 2^-126, so a p below 2^-110 may lose its lower pieces (24 bits in three of 8, the
   last 2^-16 of the first) and one below 2^-126 all of itself: 2^-109 absolute covers both;
 * a gradient: sums of those times |w| or |x|; accumulation, 128 MMAs of 2^-23 a segment (32 for
   float32, and up to 100 segments of 2^-24): 2^-16 of the sum of magnitudes (2^-17); and the
   rounding of the result, u of it (2^-25 absolute in float16).
"""

import pytest

import dense_fp32_gemm_sgemm_gb300 as sg
from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_fp32_gemm_sgemm_gb300 import build
    build.build()
    torch_cuda()


NAMES = ("f32", "bf16", "f16")


def dtype_of(name):
    torch = torch_cuda()
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def inputs(T, D, V, name, seed=0, masked=0.0, pad=0, wpad=0, weighted=False, sharp=4.0):
    """x leans towards its target's row by up to `sharp`; x and weight may be slices of wider
    tensors."""
    torch = torch_cuda()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = dtype_of(name)
    w = (torch.randn(V, D + wpad, device="cuda", generator=gen) * D ** -0.5).to(dt)[:, :D]
    y = torch.randint(V, (T,), device="cuda", generator=gen)
    x = torch.randn(T, D + pad, device="cuda", generator=gen)
    x[:, :D] += torch.rand(T, 1, device="cuda", generator=gen) * sharp * w[y].float()
    x = x.to(dt)[:, :D]
    if masked:
        y = torch.where(torch.rand(T, device="cuda", generator=gen) < masked, -100, y)
    c = None
    if weighted:
        c = (torch.rand(T, device="cuda", generator=gen) + 0.25) * 64
    return x, w, y, c


class Reference:
    """The definition in 64 bits, and the bounds above."""

    def __init__(self, x, w, y, c):
        torch = torch_cuda()
        f32, f16 = x.dtype == torch.float32, x.dtype == torch.float16
        u = torch.finfo(x.dtype).eps / 2
        T, V = x.shape[0], w.shape[0]
        counted = (y >= 0) & (y < V)
        n = int(counted.sum())
        rows = counted.nonzero()[:, 0]
        x, w = x[rows].double(), w.double()
        label = y[rows].long()
        self.share = torch.full((n,), 1 / max(n, 1), dtype=torch.float64, device=x.device)
        if c is not None:
            self.share = c[rows].double()
        s = x @ w.T
        es = (x.abs() @ w.abs().T) * (1.5 * 2 ** -18 if f32 else 2 ** -17)
        lse = torch.logsumexp(s, -1) if n else s.new_zeros(0)
        el = es.amax(-1) + 2 ** -16 + 2 ** -23 * lse.abs() if n else s.new_zeros(0)
        one = torch.arange(n, device=x.device)
        losses = lse - s[one, label]

        def spread(v, fill=0.0):
            out = torch.full((T, *v.shape[1:]), fill, dtype=torch.float64, device=v.device)
            out[rows] = v
            return out

        self.lse, self.lse_tol = spread(lse), spread(el)
        self.losses, self.losses_tol = spread(losses), spread(2 * el)
        self.loss = (self.share * losses).sum()
        self.loss_tol = (self.share.abs() * 2 * el).sum() + 2 ** -23 * self.loss.abs()
        p = torch.exp(s - lse[:, None])
        off = es + el[:, None] + 2 ** -20
        g, dg = p.clone(), p * ((2 ** -23 if f32 else 2 * u) + off) + 2.0 ** -109
        if f16 and n:
            top = self.share.abs().max() / self.share.abs().clamp(min=1e-300)
            dg += 2 ** -40 + 2 ** -39 * top[:, None]
        rest = p.clone()
        rest[one, label] = 0
        rest = rest.sum(-1)
        g[one, label] = -rest
        dg[one, label] = rest * u + p[one, label] * off[one, label] + (2 ** -39 if f16 else 0)
        g, dg = g * self.share[:, None], dg * self.share.abs()[:, None]
        acc = 2 ** -17 if f32 else 2 ** -16
        floor = 2 ** -25 if f16 else 0
        dx = g @ w
        self.dx = spread(dx)
        self.dx_tol = spread(dg @ w.abs() + acc * (g.abs() @ w.abs()) + u * dx.abs() + floor)
        self.dw = g.T @ x
        self.dw_tol = dg.T @ x.abs() + acc * (g.abs().T @ x.abs()) + u * self.dw.abs() + floor

    def check(self, out, names=("loss", "losses", "lse", "dx", "dw")):
        torch = torch_cuda()
        for name, got in zip(names, out):
            want, tol = getattr(self, name), getattr(self, name + "_tol")
            err = (got.double() - want).abs()
            assert torch.isfinite(got.double()).all(), name
            bad = err > tol
            assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} outside, worst "
                                   f"{float((err / tol.clamp(min=1e-300)).max()):.3g} of the bound")


# one token, one column, one class; tiles' borders in every dimension; several tiles; sizes whose
# reduction over the vocabulary is split
SHAPES = [(1, 1, 1), (1, 64, 2), (3, 5, 7), (64, 64, 128), (65, 63, 129), (255, 128, 256),
          (256, 65, 257), (257, 300, 1000), (300, 8, 5003), (1030, 520, 700), (40, 1024, 9000)]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("T,D,V", SHAPES)
def test_against_64_bits(T, D, V, name):
    x, w, y, c = inputs(T, D, V, name, seed=T + D, weighted=name == "f16")
    ref = Reference(x, w, y, c)
    ref.check(sg.cross_entropy(x, w, y, token_weights=c))
    ref.check(sg.cross_entropy_grad(x, w, y, token_weights=c))
    assert sg.device_error() == sg.OK


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("bits", [32, 64])
def test_masks_and_weights(name, bits):
    torch = torch_cuda()
    x, w, y, _ = inputs(700, 72, 300, name, seed=5, masked=0.4)
    y[3], y[4], y[5], y[6] = -1, 300, -(2 ** 31), 2 ** 31 - 1  # none of them counts
    gen = torch.Generator(device="cuda").manual_seed(6)
    c = torch.randn(700, device="cuda", generator=gen)  # of both signs, some zero
    c[::7] = 0
    if bits == 32:
        y = y.int()
    else:
        y[7] = 2 ** 40
    for weights in (None, c):
        Reference(x, w, y, weights).check(sg.cross_entropy_grad(x, w, y, token_weights=weights))


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("T", [70, 1500])  # the two ways that tokens are selected
def test_what_does_not_count_is_not_read(name, T):
    """Infinities and NaN in masked rows, in their weights, and behind the rows' ends."""
    torch = torch_cuda()
    x, w, y, c = inputs(T, 40, 200, name, seed=7, masked=0.5, pad=9, wpad=16, weighted=True)
    hidden = y < 0
    wide_x, wide_w = x._base, w._base
    wide_x[:, 40:] = float("nan")
    wide_w[:, 40:] = float("inf")
    x[hidden] = float("nan")
    x[hidden.nonzero()[0]] = float("inf")
    c[hidden] = float("nan")
    out = sg.cross_entropy_grad(x, w, y, token_weights=c)
    Reference(x, w, y, c).check(out)
    assert not out.dx[hidden].any() and not out.losses[hidden].any() and not out.lse[hidden].any()


@pytest.mark.parametrize("name", NAMES)
def test_no_token_counts(name):
    torch = torch_cuda()
    x, w, y, _ = inputs(130, 40, 200, name)
    y.fill_(-100)
    x.fill_(float("nan"))
    for c in (None, torch.ones(130, device="cuda")):
        out = sg.cross_entropy_grad(x, w, y, token_weights=c)
        for t in out:
            assert not t.any()
    out = sg.cross_entropy_grad(x[:0], w, y[:0])
    assert out.dx.shape == (0, 40) and float(out.loss) == 0 and not out.dweight.any()
    assert float(sg.cross_entropy(x[:0], w, y[:0]).loss) == 0


@pytest.mark.parametrize("name", NAMES)
def test_strides_and_outputs_given(name):
    """Slices of wider tensors for all of x, weight, dx and dweight, at odd offsets: the same values
    as from contiguous ones to the bit, and nothing outside is touched."""
    torch = torch_cuda()
    x, w, y, c = inputs(333, 77, 501, name, seed=9, masked=0.2, pad=5, wpad=3)
    want = sg.cross_entropy_grad(x.contiguous(), w.contiguous(), y)
    dx = torch.full((333, 90), 7.0, device="cuda", dtype=x.dtype)
    dw = torch.full((501, 81), 7.0, device="cuda", dtype=x.dtype)
    got = sg.cross_entropy_grad(x, w, y, dx=dx[:, 3:80], dweight=dw[:, 1:78])
    assert got.dx.data_ptr() == dx[:, 3:].data_ptr()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    assert (dx[:, :3] == 7).all() and (dx[:, 80:] == 7).all()
    assert (dw[:, :1] == 7).all() and (dw[:, 78:] == 7).all()
    # a shifted, but contiguous input: the address is not 16-byte aligned
    flat = torch.empty(501 * 77 + 1, device="cuda", dtype=x.dtype)[1:]
    w1 = flat.view(501, 77).copy_(w)
    assert torch.equal(sg.cross_entropy_grad(x, w1, y).dx, want.dx)


@pytest.mark.parametrize("name", NAMES)
def test_one_gradient_alone(name):
    torch = torch_cuda()
    x, w, y, c = inputs(600, 136, 1100, name, seed=10, masked=0.1)
    both = sg.cross_entropy_grad(x, w, y)
    a = sg.cross_entropy_grad(x, w, y, need_dweight=False)
    b = sg.cross_entropy_grad(x, w, y, need_dx=False)
    assert a.dweight is None and b.dx is None
    assert torch.equal(b.dweight, both.dweight)
    Reference(x, w, y, c).check((a.loss, a.losses, a.lse, a.dx), ("loss", "losses", "lse", "dx"))
    none = sg.cross_entropy_grad(x, w, y, need_dx=False, need_dweight=False)
    assert torch.equal(none.losses, sg.cross_entropy(x, w, y).losses)


@pytest.mark.parametrize("name", NAMES)
def test_confident_and_far_tokens(name):
    """Logits of hundreds: p of the target near one, whose gradient is what is left of p - 1, and
    targets whose p underflows."""
    x, w, y, c = inputs(200, 96, 400, name, seed=11, sharp=0.0)
    x = (x.float() + 18 * w[y].float()).to(x.dtype)  # about 18 above the others
    Reference(x, w, y, c).check(sg.cross_entropy_grad(x, w, y))
    far = (x.float() * 20).to(x.dtype)
    far_y = y.roll(1)
    Reference(far, w, far_y, c).check(sg.cross_entropy_grad(far, w, far_y))


def test_infinite_logits():
    """-inf logits have no weight; a row of NaN is a NaN of its own and no other's."""
    torch = torch_cuda()
    x, w, y, _ = inputs(70, 64, 600, "bf16", seed=12, sharp=0.0)
    x[:, 0] = 1.0
    w[:, 0] = 0.0
    w[130:470, 0] = float("-inf")  # whole blocks of columns and parts
    y = torch.where((y >= 130) & (y < 470), y % 130, y)
    keep = torch.cat([w[:130], w[470:]])
    got = sg.cross_entropy(x, w, y)
    want = sg.cross_entropy(x, keep, torch.where(y >= 470, y - 340, y))
    assert torch.allclose(got.lse, want.lse, rtol=2 ** -20, atol=2 ** -16)
    w[:, 0] = 0.0
    x[5, 3] = float("nan")
    got = sg.cross_entropy_grad(x, w, y, need_dweight=False)
    clean = x.clone()
    clean[5, 3] = 0
    fine = sg.cross_entropy_grad(clean, w, y, need_dweight=False)
    others = torch.arange(70, device="cuda") != 5
    assert torch.isnan(got.losses[5]) and torch.isnan(got.dx[5]).all()
    assert torch.equal(got.losses[others], fine.losses[others])
    assert torch.equal(got.dx[others], fine.dx[others])


@pytest.mark.parametrize("name", ["bf16", "f32"])
def test_chunks_of_tokens(name):
    """So many logits that tokens are worked through in chunks (2 GiB of them at a time): dweight
    is summed over the chunks. Against 64 bits on sampled rows and classes."""
    torch = torch_cuda()
    T, D, V = (1500, 24, 1 << 20) if name == "bf16" else (600, 24, 1 << 20)
    x, w, y, _ = inputs(T, D, V, name, seed=13, masked=0.1, sharp=8.0)
    y[:40] = torch.arange(40, device="cuda") % 8  # classes with several tokens, in the first chunk
    y[-40:] = torch.arange(40, device="cuda") % 8  # and the last
    out = sg.cross_entropy_grad(x, w, y)
    again = sg.cross_entropy_grad(x, w, y)
    for a, b in zip(out, again):
        assert torch.equal(a, b)
    classes = torch.cat([torch.arange(16, device="cuda"), torch.tensor([V - 1, V - 129], device="cuda"),
                         torch.arange(5000, V, 30011, device="cuda")])
    u = torch.finfo(x.dtype).eps / 2
    rows = ((y >= 0) & (y < V)).nonzero()[:, 0]
    dw = torch.zeros(len(classes), D, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(dw)
    size = torch.zeros_like(dw)
    for part in rows.split(64):
        xs = x[part].double()
        s = xs @ w.double().T
        es = (xs.abs() @ w.double().abs().T).amax(-1) * 2 ** -17
        lse = torch.logsumexp(s, -1)
        el = es + 2 ** -16 + 2 ** -23 * lse.abs()
        assert ((out.lse[part] - lse).abs() <= el).all()
        p = torch.exp(s - lse[:, None])[:, classes]
        hit = y[part][:, None] == classes
        g = torch.where(hit, p - 1, p) / len(rows)
        dg = (p * (2 * u + es + el + 2 ** -20)[:, None] + hit * u * (1 - p)) / len(rows)
        dw += g.T @ xs
        tol += dg.T @ xs.abs()
        size += g.abs().T @ xs.abs()
    tol += 2 ** -16 * size + u * dw.abs()
    assert ((out.dweight[classes].double() - dw).abs() <= tol).all()


def test_chunks_of_tokens_without_gradients():
    """The statistics alone of very many columns are bounded too."""
    torch = torch_cuda()
    T, V = 17000, 1 << 20
    x, w, y, _ = inputs(T, 8, V, "bf16", seed=14)
    out = sg.cross_entropy(x, w, y)
    part = torch.tensor([0, 1, 16383, 16384, 16999], device="cuda")
    alone = sg.cross_entropy(x[part], w, y[part])
    # 64 columns a block there, 128 here: sums in another order
    assert torch.allclose(out.lse[part], alone.lse, rtol=2 ** -21, atol=2 ** -17)
    mean = out.losses.double().mean()
    assert abs(float(out.loss) - float(mean)) <= 2 ** -22 * abs(float(mean))


def test_offsets_beyond_31_bits():
    """2.4e9 elements of x: the last rows' gradients, and a class of their own at the end."""
    torch = torch_cuda()
    T, D, V = 600001, 4096, 256
    gen = torch.Generator(device="cuda").manual_seed(30)
    x = torch.empty(T, D, device="cuda", dtype=torch.bfloat16)
    x.view(-1, 4096)[:] = 0
    x[-700:] = torch.randn(700, D, device="cuda", generator=gen).to(torch.bfloat16)
    w = (torch.randn(V, D, device="cuda", generator=gen) * D ** -0.5).to(torch.bfloat16)
    y = torch.full((T,), -100, device="cuda")
    y[-700:] = torch.randint(V, (700,), device="cuda", generator=gen)
    y[:100000] = 3  # rows of zeros: equal logits, no gradient of the weights
    out = sg.cross_entropy_grad(x, w, y)
    tail = Reference(x[-700:], w, y[-700:], torch.full((700,), 1 / 100700, device="cuda"))
    tail.check((out.losses[-700:], out.lse[-700:], out.dx[-700:], out.dweight),
               ("losses", "lse", "dx", "dw"))
    assert (out.lse[:100000] - 8 * 0.6931471805599453).abs().max() <= 2 ** -16
    assert not out.dx[100000:-700].any()


def test_rows_gigabytes_apart():
    """Weights and their gradient with rows 2^31 bytes apart; without tokens, the zeros there too."""
    torch = torch_cuda()
    T, D, V, pitch = 70, 96, 3, 2 ** 30 + 64
    x, w, y, _ = inputs(T, D, V, "bf16")
    expected = sg.cross_entropy_grad(x, w, y)
    wide = torch.empty_strided((V, D), (pitch, 1), device="cuda", dtype=torch.bfloat16)
    wide.copy_(w)
    dw = torch.empty_strided((V, D), (pitch, 1), device="cuda", dtype=torch.bfloat16)
    out = sg.cross_entropy_grad(x, wide, y, dweight=dw)
    for got, want in zip(out, expected):
        assert torch.equal(got, want)
    dw.fill_(float("nan"))
    sg.cross_entropy_grad(x[:0], wide, y[:0], dweight=dw)
    assert not dw.any()


def test_gradient_against_differences():
    """Central differences of the float32 loss along random directions against the gradients. Each
    loss is off by 2^-18 at most here; what the step itself costs (h^2 / 6 of the third derivative) is
    how far the same differences in 64 bits are from the slope in 64 bits."""
    torch = torch_cuda()
    x, w, y, c = inputs(90, 48, 333, "f32", seed=15, masked=0.2)
    gen = torch.Generator(device="cuda").manual_seed(16)
    out = sg.cross_entropy_grad(x, w, y)

    def exact(x, w):
        rows = (y >= 0).nonzero()[:, 0]
        s = x[rows].double() @ w.double().T
        return (torch.logsumexp(s, -1) - s.gather(1, y[rows][:, None])[:, 0]).mean()

    for which, t, grad in (("x", x, out.dx), ("w", w, out.dweight)):
        d = torch.randn(t.shape, device="cuda", generator=gen)
        h = 2.0 ** -5 if which == "x" else 2.0 ** -6
        hi, lo = t + h * d, t - h * d
        args = [((v, w) if which == "x" else (x, v)) for v in (hi, lo)]
        got = sum(k * float(sg.cross_entropy(a, b, y).loss) for k, (a, b) in zip((1, -1), args))
        sure = sum(k * float(exact(a, b)) for k, (a, b) in zip((1, -1), args))
        # the step as taken, rounded to float32
        slope = float((grad.double() * ((hi.double() - lo.double()))).sum())
        assert abs(got - sure) <= 2 * 2 ** -18
        leaf = t.double().requires_grad_()
        exact(*((leaf, w) if which == "x" else (x, leaf))).backward()
        true = float((leaf.grad * (hi.double() - lo.double())).sum())
        assert abs(slope - sure) <= abs(true - sure) + 2 * 2 ** -18


@pytest.mark.parametrize("name", NAMES)
def test_graphs_on_two_streams(name):
    """Two captured calls replayed at the same time, with new inputs, against direct calls."""
    torch = torch_cuda()
    cases = [inputs(T, 200, 3000, name, seed=17 + T, masked=0.3) for T in (500, 1100)]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in cases]
    for (x, w, y, c) in cases:
        sg.cross_entropy_grad(x, w, y)
    torch.cuda.synchronize()
    for (x, w, y, c), s in zip(cases, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(sg.cross_entropy_grad(x, w, y))
        graphs.append(g)
    for (x, w, y, c) in cases:
        x.mul_(1.25)
        y.copy_(torch.where(y < 0, 5, torch.where(y % 3 == 0, -100, y)))  # other tokens count
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (x, w, y, c), out in zip(cases, outs):
        for a, b in zip(out, sg.cross_entropy_grad(x, w, y)):
            assert torch.equal(a, b)
    assert sg.device_error() == sg.OK


def test_two_streams_at_once():
    torch = torch_cuda()
    cases = [inputs(T, 256, 4000, "bf16", seed=20 + T) for T in (300, 900)]
    want = [sg.cross_entropy_grad(x, w, y) for x, w, y, c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, (s, (x, w, y, c)) in enumerate(zip(streams, cases)):
            got[i].append(sg.cross_entropy_grad(x, w, y, stream=s))
    torch.cuda.synchronize()
    for a, runs in zip(want, got):
        for b in runs:
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_refusals_of_the_binding():
    torch = torch_cuda()
    x, w, y, _ = inputs(8, 16, 30, "bf16")
    c = torch.ones(8, device="cuda")
    for bad in (lambda: sg.cross_entropy(x, w.float(), y), lambda: sg.cross_entropy(x[:, :15], w, y),
                lambda: sg.cross_entropy(x, w, y[:7]), lambda: sg.cross_entropy(x, w, y.float()),
                lambda: sg.cross_entropy(x, w, y[::2].repeat(1, 2)),
                lambda: sg.cross_entropy(x.T, w, y), lambda: sg.cross_entropy(x.double(), w, y),
                lambda: sg.cross_entropy(x, w[0], y), lambda: sg.cross_entropy(x, w, y.cpu()),
                lambda: sg.cross_entropy(x, w, y, token_weights=c[:7]),
                lambda: sg.cross_entropy(x, w, y, token_weights=c.double()),
                lambda: sg.cross_entropy_grad(x, w, y, dx=torch.empty_like(x).float()),
                lambda: sg.cross_entropy_grad(x, w, y, dweight=w.T),
                lambda: sg.cross_entropy_grad(x, w, y, dx=torch.empty(8, 8, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(sg.SgemmError):  # an output that is an input
        sg.cross_entropy_grad(x, w, y, dx=x)
    with pytest.raises(sg.SgemmError):
        sg.cross_entropy_grad(x, w, y, dx=torch.as_strided(w, (8, 16), (16, 1)))

"""Cases of the training operators: the cross entropy of an output head, with its gradients,
and updates orthogonalised by Newton-Schulz products.

Each case can run in a plain form (elementary torch operations in 32 bits) or, with
``own`` set, through the library's own entry points. ``exact`` gives the same outputs
from the definitions in 64 bits.
"""

import math

import torch

own = False

DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
BYTES = {"float32": 4, "bfloat16": 2, "float16": 2}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7
EXACT_FLOPS = 1e13  # beyond this the 64-bit form takes too long


def listed():
    return [
        # One token scored against a small vocabulary: latency is everything.
        loss_case("score-token", "bfloat16", 1, 512, 4096),
        # A prompt scored token by token against a large vocabulary.
        loss_case("score-prompt", "bfloat16", 2048, 4096, 65536),
        # A training step's head in a small model: launches and latency count.
        loss_case("head-small", "bfloat16", 256, 512, 8192, grad=True),
        # An ordinary one, some of its tokens padding.
        loss_case("head-medium", "bfloat16", 4096, 2048, 32768, grad=True, masked=0.2),
        # Odd sizes, x a slice of a wider tensor, weights for each token that carry a loss
        # scale, and most tokens masked, as a prompt's are in fine-tuning.
        loss_case("head-ragged", "float16", 1111, 777, 10007, grad=True, masked=0.6, weighted=True,
                  pad=5),
        # The library's own type.
        loss_case("head-f32", "float32", 1024, 1024, 32000, grad=True),
        # A long batch through a large head.
        loss_case("head-large", "bfloat16", 8192, 4096, 65536, grad=True),
        # An update of one small projection: latency again.
        update_case("update-small", "bfloat16", 1, 256, 256),
        # A square projection.
        update_case("update-square", "bfloat16", 1, 4096, 4096),
        # A tall matrix of odd sizes in the library's own type.
        update_case("update-ragged", "float32", 1, 2731, 1001),
        # The experts of a layer, one stack.
        update_case("update-stack", "float16", 16, 512, 2048),
        # A large matrix.
        update_case("update-large", "bfloat16", 1, 6144, 8192),
    ]


def loss_case(name, dtype, t, d, v, grad=False, masked=0.0, weighted=False, pad=0):
    return named(name, {"op": "loss", "dtype": dtype, "t": t, "d": d, "v": v, "grad": grad,
                        "masked": masked, "weighted": weighted, "pad": pad})


def update_case(name, dtype, e, m, n):
    return named(name, {"op": "update", "dtype": dtype, "e": e, "m": m, "n": n})


def named(name, case):
    return case if name is None else {"name": name, **case}


def draw(rng):
    def size(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))

    # 32-bit types are multiplied in pieces, so that they get smaller sizes
    while True:
        dtype = rng.choice(["float32", "bfloat16", "bfloat16", "float16"])
        if rng.random() < 0.5:
            grad = rng.random() < 0.7
            t, d, v = size(1, 8192), size(128, 4096), size(1000, 65536)
            if t * d * v > (2 ** 41 if dtype != "float32" else 2 ** 37):
                continue
            return loss_case(None, dtype, t, d, v, grad, rng.choice([0.0, 0.2, 0.6]),
                             dtype == "float16" or rng.random() < 0.3, rng.choice([0, 0, 8, 3]))
        m, n = size(64, 8192), size(64, 8192)
        e = rng.choice([1, 1, size(2, 32)])
        if e * m * n * min(m, n) > (2 ** 38 if dtype == "bfloat16" else 2 ** 36):
            continue
        return update_case(None, dtype, e, m, n)


# ---- inputs -------------------------------------------------------------------------

def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def loss_inputs(case, seed):
    """Hidden states that lean towards the target's row of the head, some tokens much more
    than others, as a model in training has them. Masked tokens have the target -100."""
    gen = generator(seed)
    dtype = DTYPES[case["dtype"]]
    t, d, v = case["t"], case["d"], case["v"]
    weight = normal(gen, v, d).mul_(d ** -0.5).to(dtype)
    target = torch.randint(v, (t,), generator=gen, device="cuda")
    lean = torch.rand(t, 1, generator=gen, device="cuda") * 12
    x = normal(gen, t, d + case["pad"])
    x[:, :d] += lean * weight[target].float()
    x = x.to(dtype)[:, :d]
    if case["masked"]:
        hidden = torch.rand(t, generator=gen, device="cuda") < case["masked"]
        target = torch.where(hidden, torch.full_like(target, -100), target)
    c = None
    if case["weighted"]:
        c = (0.5 + torch.rand(t, generator=gen, device="cuda")) * 256
    return x, weight, target, c


def update_inputs(case, seed):
    """A gradient averaged over steps: a few strong directions over noise."""
    gen = generator(seed)
    e, m, n = case["e"], case["m"], case["n"]
    rank = max(1, min(m, n) // 64)
    g = normal(gen, e, m, n)
    g += (4 * rank ** -0.5) * (normal(gen, e, m, rank) @ normal(gen, e, rank, n))
    g = g.mul_(1e-3).to(DTYPES[case["dtype"]])
    return g[0] if e == 1 else g


def prepare(case, seed):
    if case["op"] == "loss":
        x, weight, target, c = loss_inputs(case, seed)
        return {"case": case, "x": x, "weight": weight, "target": target, "c": c}
    return {"case": case, "g": update_inputs(case, seed)}


# ---- the operators ------------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        return run_own(state, case)
    if case["op"] == "loss":
        return plain_loss(state["x"], state["weight"], state["target"], state["c"], case["grad"])
    return plain_update(state["g"])


def run_own(state, case):
    import dense_fp32_gemm_sgemm_gb300 as sg

    if case["op"] == "loss":
        call = sg.cross_entropy_grad if case["grad"] else sg.cross_entropy
        return tuple(call(state["x"], state["weight"], state["target"], token_weights=state["c"]))
    return sg.orthogonalize(state["g"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)


def plain_loss(x, weight, target, c, grad):
    """Losses by pieces of the vocabulary with a running maximum and sum; gradients by the
    same pieces, their logits computed again."""
    dtype, (t, _), v = x.dtype, x.shape, weight.shape[0]
    counted = (target >= 0) & (target < v)
    x = torch.where(counted[:, None], x.float(), torch.zeros((), device=x.device))
    if c is None:
        c = 1 / counted.sum().clamp(min=1).float().expand(t)
    c = torch.where(counted, c, torch.zeros((), device=x.device))
    piece = 8192
    top = torch.full((t,), -math.inf, device=x.device)
    total = torch.zeros(t, device=x.device)
    picked = torch.zeros(t, device=x.device)
    for first in range(0, v, piece):
        s = x @ weight[first:first + piece].float().mT
        new = torch.maximum(top, s.amax(-1))
        total = total * torch.exp(top - new) + torch.exp(s - new[:, None]).sum(-1)
        top = new
        here = (target >= first) & (target < first + s.shape[1])
        index = (target - first).clamp(0, s.shape[1] - 1)
        picked = torch.where(here, s.gather(1, index[:, None])[:, 0], picked)
    zero = torch.zeros((), device=x.device)
    lse = torch.where(counted, top + torch.log(total), zero)
    losses = torch.where(counted, lse - picked, zero)
    loss = (c * losses).sum()
    if not grad:
        return loss, losses, lse
    dx = torch.zeros_like(x)
    dweight = torch.empty(weight.shape, dtype=dtype, device=x.device)
    for first in range(0, v, piece):
        w = weight[first:first + piece].float()
        s = x @ w.mT - lse[:, None]
        label = target[:, None] == torch.arange(first, first + w.shape[0], device=x.device)
        g = torch.where(label, torch.expm1(s), torch.exp(s)) * c[:, None]
        dx += g @ w
        dweight[first:first + piece] = (g.mT @ x).to(dtype)
    return loss, losses, lse, dx.to(dtype), dweight


def plain_update(g):
    a, b, c = COEFFICIENTS
    tall = g.shape[-2] > g.shape[-1]
    x = g.float()
    x = x.mT if tall else x
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + EPS)
    for _ in range(STEPS):
        gram = x @ x.mT
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return (x.mT if tall else x).to(g.dtype).contiguous()


# ---- the definitions in 64 bits -----------------------------------------------------

def exact(case, seed):
    if 4 * work(case)["flops"] / 3 > EXACT_FLOPS:
        return None
    if case["op"] == "loss":
        return exact_loss(*loss_inputs(case, seed), case["grad"])
    g = update_inputs(case, seed).double()
    if g.dim() == 2:
        return exact_update(g)
    return torch.stack([exact_update(m) for m in g])


def exact_loss(x, weight, target, c, grad):
    """Token by token in blocks, each with its whole row of logits."""
    t, v = x.shape[0], weight.shape[0]
    w = weight.double()
    losses = torch.zeros(t, dtype=torch.float64, device=x.device)
    lse = torch.zeros_like(losses)
    dx = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    dweight = torch.zeros_like(w)
    index = torch.nonzero((target >= 0) & (target < v))[:, 0]
    share = torch.zeros(t, dtype=torch.float64, device=x.device)
    if len(index):
        share[index] = 1 / len(index) if c is None else c[index].double()
    for rows in index.split(1024):
        if not len(rows):
            continue
        s = x[rows].double() @ w.T
        one = torch.arange(len(rows), device=x.device)
        lse[rows] = torch.logsumexp(s, -1)
        losses[rows] = lse[rows] - s[one, target[rows]]
        if grad:
            p = torch.softmax(s, -1)
            # p - 1 of the target: minus the others' sum
            p[one, target[rows]] = 0
            p[one, target[rows]] = -p.sum(-1)
            p *= share[rows, None]
            dx[rows] = p @ w
            dweight += p.T @ x[rows].double()
    loss = (share * losses).sum()
    return (loss, losses, lse, dx, dweight) if grad else (loss, losses, lse)


def exact_update(g):
    """With the Gram matrix of the smaller side, from the left or from the right."""
    a, b, c = (torch.tensor(f, dtype=torch.float64, device=g.device) for f in COEFFICIENTS)
    x = g / (torch.linalg.vector_norm(g) + EPS)
    eye = torch.eye(min(g.shape), dtype=torch.float64, device=g.device)
    for _ in range(STEPS):
        if g.shape[0] > g.shape[1]:
            gram = x.T @ x
            x = x @ (a * eye + gram @ (b * eye + c * gram))
        else:
            gram = x @ x.T
            x = (a * eye + gram @ (b * eye + c * gram)) @ x
    return x


# ---- what a pass cannot do without --------------------------------------------------

def work(case):
    size = BYTES[case["dtype"]]
    if case["op"] == "loss":
        t, d, v = case["t"], case["d"], case["v"]
        lively = t * (1 - case["masked"])
        # read x of the tokens that count, the head, targets and weights; write the losses
        moved = size * (lively * d + v * d) + t * (8 + 8 + (4 if case["weighted"] else 0))
        if case["grad"]:
            # write both gradients; three products
            return {"bytes": moved + size * (t * d + v * d), "flops": 6 * lively * d * v}
        return {"bytes": moved, "flops": 2 * lively * d * v}
    e, m, n = case["e"], case["m"], case["n"]
    low, high = min(m, n), max(m, n)
    # a step: half of a symmetric product of each kind, and a whole one
    step = low * low * high + low ** 3 + 2 * low * low * high
    return {"bytes": 2 * size * e * m * n, "flops": STEPS * e * step}

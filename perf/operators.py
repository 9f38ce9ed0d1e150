"""Cases of the 4-bit operators: quantisation, few-row products and the mixture-of-experts layer.

Each case can run in a plain form (elementary torch operations in 32 bits) or, with
``own`` set, through the library's own entry points. ``exact`` gives the same outputs
from the definitions in 64 bits.
"""

import math

import torch

own = False

DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
BYTES = {"float32": 4, "bfloat16": 2, "float16": 2}


def listed():
    return [
        # Weights quantised when a checkpoint is loaded, and read back for a product with
        # many rows: the library's largest square matrix ...
        quantize_case("quantize-square", "float32", 8192, 8192, 128),
        # ... and odd sizes, rows stored per output column, with zero points.
        quantize_case("quantize-ragged", "bfloat16", 4095, 4097, 32, zeros=True, transposed=True),
        # One token through a small projection: latency is everything.
        matmul_case("row-small", "bfloat16", 1, 512, 512, 64),
        # One token in the library's own type through an ordinary projection.
        matmul_case("row-f32", "float32", 1, 6144, 4096, 128),
        # One token through a large square projection.
        matmul_case("row-large", "bfloat16", 1, 8192, 8192, 128),
        # A few tokens at odd sizes, as a slice of a wider tensor, with an imported
        # checkpoint's float16 scales and zero points in the smallest groups.
        matmul_case("rows-ragged", "float16", 5, 8191, 4097, 32, zeros=True, scale="float16", pad=9),
        # A batch of sixteen sequences, one token each.
        matmul_case("rows-batch", "bfloat16", 16, 8192, 6144, 64),
        # Sixty-four tokens through an output head: more weights than any cache holds.
        matmul_case("rows-head", "bfloat16", 64, 8192, 65536, 128),
        # One token through a small layer of experts: latency again.
        moe_case("moe-small", "bfloat16", 1, 512, 512, 8, 2, 64),
        # One token through a large layer: eight experts of sixty-four are read.
        moe_case("moe-token", "bfloat16", 1, 4096, 2048, 64, 8, 128),
        # A part-filled batch at odd sizes in the library's own type.
        moe_case("moe-ragged", "float32", 7, 1000, 777, 12, 3, 32, zeros=True, masked=True),
        # A full batch: nearly every expert is read, each by several tokens.
        moe_case("moe-batch", "bfloat16", 64, 4096, 2048, 64, 8, 128),
    ]


def quantize_case(name, dtype, n, k, group, zeros=False, transposed=False):
    return named(name, {"op": "quantize", "dtype": dtype, "n": n, "k": k, "group": group,
                        "zeros": zeros, "transposed": transposed})


def matmul_case(name, dtype, m, n, k, group, zeros=False, scale="bfloat16", pad=0):
    return named(name, {"op": "matmul", "dtype": dtype, "m": m, "n": n, "k": k, "group": group,
                        "zeros": zeros, "scale": scale, "pad": pad})


def moe_case(name, dtype, t, d, f, e, top, group, zeros=False, masked=False, renorm=True):
    return named(name, {"op": "moe", "dtype": dtype, "t": t, "d": d, "f": f, "e": e, "top": top,
                        "group": group, "zeros": zeros, "masked": masked, "renorm": renorm})


def named(name, case):
    return case if name is None else {"name": name, **case}


def draw(rng):
    def size(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))

    op = rng.choice(["quantize", "matmul", "matmul", "moe", "moe"])
    dtype = rng.choice(["float32", "bfloat16", "bfloat16", "float16"])
    group = rng.choice([32, 64, 128])
    zeros = rng.random() < 0.4
    if op == "quantize":
        return quantize_case(None, dtype, size(512, 8192), size(512, 8192), group, zeros,
                             rng.random() < 0.5)
    if op == "matmul":
        return matmul_case(None, dtype, size(1, 64), size(256, 8192), size(256, 65536), group, zeros,
                           rng.choice(["bfloat16", "float16"]), rng.choice([0, 0, 8, 3]))
    e = size(4, 64)
    return moe_case(None, dtype, size(1, 64), size(256, 4096), size(256, 2048), e,
                    rng.randint(1, min(8, e)), group, zeros, rng.random() < 0.3,
                    rng.random() < 0.7)


# ---- inputs -------------------------------------------------------------------------

def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def weights(gen, n, *shape):
    """Normal weights whose products keep the size of their inputs, n terms a sum."""
    return normal(gen, *shape).mul_(n ** -0.5)


def activations(gen, rows, cols, dtype):
    """Normal rows, with one column in about a hundred eight times as large, as the
    residual stream of a language model has them."""
    x = normal(gen, rows, cols)
    large = torch.rand(cols, generator=gen, device="cuda") < 0.01
    return (x * torch.where(large, 8.0, 1.0)).to(dtype)


def quantized(gen, case, stack, n, k, scale):
    """A random matrix (or a stack) in codes, scales and zero points."""
    w = weights(gen, n, *stack, n, k)
    codes, scales, zeros = codes_of(w, case["group"], case["zeros"], scale)
    return {"codes": codes, "scales": scales, "zeros": zeros, "group": case["group"]}


def packed(q):
    """The library's form of the same matrix, laid out once as a program does on loading."""
    import dense_fp32_gemm_sgemm_gb300 as sg

    return sg.q4_pack(q["codes"], q["scales"], q["zeros"], group=q["group"])


def prepare(case, seed):
    gen = generator(seed)
    dtype = DTYPES[case["dtype"]]
    state = {"case": case}
    if case["op"] == "quantize":
        shape = (case["k"], case["n"]) if case["transposed"] else (case["n"], case["k"])
        state["b"] = weights(gen, case["n"], *shape).to(dtype)
        return state
    if case["op"] == "matmul":
        a = activations(gen, case["m"], case["n"] + case["pad"], dtype)
        state["a"] = a[:, :case["n"]]
        w = quantized(gen, case, (), case["n"], case["k"], DTYPES[case["scale"]])
        state["w"] = packed(w) if own else w
        return state
    t, d, f, e = case["t"], case["d"], case["f"], case["e"]
    state["x"] = activations(gen, t, d, dtype)
    state["live"] = None
    if case["masked"]:
        state["live"] = torch.rand(t, generator=gen, device="cuda") < 0.7
    router = weights(gen, d, e, d).to(dtype)
    mats = []
    for n, k in ((d, f), (d, f), (f, d)):
        w = quantized(gen, case, (e,), n, k, torch.bfloat16)
        mats.append(packed(w) if own else w)
        del w
    if own:
        import dense_fp32_gemm_sgemm_gb300 as sg

        state["layer"] = sg.MoeLayer(router, *mats, top_k=case["top"], renormalize=case["renorm"])
    else:
        state["router"], state["gate"], state["up"], state["down"] = router, *mats
    return state


# ---- the operators ------------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        return run_own(state, case)
    if case["op"] == "quantize":
        b = state["b"].float()
        b = b.mT.contiguous() if case["transposed"] else b
        codes, scales, zeros = codes_of(b, case["group"], case["zeros"], torch.bfloat16)
        return values_of(codes, scales, zeros, case["group"])
    if case["op"] == "matmul":
        return (state["a"].float() @ values_of(**state["w"])).to(state["a"].dtype)
    return plain_moe(state, case)


def run_own(state, case):
    import dense_fp32_gemm_sgemm_gb300 as sg

    if case["op"] == "quantize":
        w = sg.q4_quantize(state["b"], group=case["group"], zeros=case["zeros"],
                           transposed=case["transposed"])
        return sg.q4_dequantize(w)
    if case["op"] == "matmul":
        return sg.q4_matmul(state["a"], state["w"])
    return state["layer"](state["x"], live=state["live"])


def grouped(w, group):
    """(..., n, k) as (..., groups, group, k), the last group filled up with zeros."""
    n, k = w.shape[-2:]
    fill = -n % group
    w = torch.nn.functional.pad(w, (0, 0, 0, fill)) if fill else w
    return w.reshape(*w.shape[:-2], (n + fill) // group, group, k)


def codes_of(w, group, with_zeros, scale_dtype):
    """4-bit codes (0..15) of float32 w (..., n, k), with a scale and, where asked for, a
    zero point for each group of rows in a column."""
    n = w.shape[-2]
    g = grouped(w, group)
    # divisors as tensors: a number would be turned into a product with its reciprocal
    if with_zeros:
        fifteen = torch.full((), 15.0, device=w.device)
        hi, lo = g.amax(-2).clamp(min=0), g.amin(-2).clamp(max=0)
        scales = (hi / fifteen - lo / fifteen).to(scale_dtype)
    else:
        scales = (g.abs().amax(-2) / torch.full((), 7.0, device=w.device)).to(scale_dtype)
    s = scales.float()
    some = s > 0
    s = torch.where(some, s, torch.ones_like(s))
    if with_zeros:
        zeros = torch.where(some, torch.round(-lo / s).clamp(0, 15), torch.zeros_like(s))
        q = (torch.round(g / s.unsqueeze(-2)) + zeros.unsqueeze(-2)).clamp_(0, 15)
        zeros = zeros.to(torch.uint8)
    else:
        zeros = None
        q = torch.round(g / s.unsqueeze(-2)).clamp_(-8, 7).add_(8)
    q = torch.where(some.unsqueeze(-2), q, torch.full((), 0.0 if with_zeros else 8.0, device=w.device))
    q = q.to(torch.uint8).flatten(-3, -2)[..., :n, :]
    return q.contiguous(), scales, zeros


def values_of(codes, scales, zeros, group):
    """The float32 values that codes, scales and zero points stand for."""
    n = codes.shape[-2]
    z = 8.0 if zeros is None else zeros.float().repeat_interleave(group, -2)[..., :n, :]
    return (codes.float() - z) * scales.float().repeat_interleave(group, -2)[..., :n, :]


def picked(w, index):
    """The matrices of a stack that `index` names."""
    return {"codes": w["codes"][index], "scales": w["scales"][index],
            "zeros": None if w["zeros"] is None else w["zeros"][index], "group": w["group"]}


def routing(logits, top, renorm, live):
    """The chosen experts in ascending order and their weights; ties go to the lowest index."""
    p = torch.exp(logits - logits.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    ids = torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :top].sort(-1).values
    w = p.gather(1, ids)
    if renorm:
        w = w / w.sum(-1, keepdim=True)
    if live is not None:
        w = torch.where(live[:, None], w, torch.zeros_like(w))
        ids = torch.where(live[:, None], ids, torch.full_like(ids, -1))
    return ids, w


def silu(g):
    return g / (1 + torch.exp(-g))


def plain_moe(state, case):
    x, live = state["x"].float(), state["live"]
    t, e, top = case["t"], case["e"], case["top"]
    ids, w = routing(x @ state["router"].float().mT, top, case["renorm"], live)
    if t * top <= e:
        # few choices: every chosen expert by itself
        index = ids.clamp(min=0).flatten()
        gate, up, down = (values_of(**picked(state[m], index)) for m in ("gate", "up", "down"))
        rows = x.repeat_interleave(top, 0).unsqueeze(1)
        h = silu(rows @ gate) * (rows @ up)
        y = ((h @ down).reshape(t, top, -1) * w.unsqueeze(-1)).sum(1)
    else:
        # many: every expert for every token, the weights of those not chosen zero
        share = torch.zeros(t, e + 1, device=x.device).scatter(1, torch.where(ids < 0, e, ids), w)[:, :e]
        h = silu(x @ values_of(**state["gate"]))
        h = h * (x @ values_of(**state["up"])) * share.mT.unsqueeze(-1)
        y = (h @ values_of(**state["down"])).sum(0)
    return y.to(state["x"].dtype), ids.to(torch.int32), w


# ---- the definitions in 64 bits -----------------------------------------------------

def exact(case, seed):
    gen = generator(seed)
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "quantize":
        shape = (case["k"], case["n"]) if case["transposed"] else (case["n"], case["k"])
        b = weights(gen, case["n"], *shape).to(dtype).double()
        return exact_quantized(b.mT if case["transposed"] else b, case["group"], case["zeros"])
    if case["op"] == "matmul":
        a = activations(gen, case["m"], case["n"] + case["pad"], dtype)[:, :case["n"]].double()
        w = quantized(gen, case, (), case["n"], case["k"], DTYPES[case["scale"]])
        return a @ exact_values(w, slice(None))
    return exact_moe(case, gen, dtype)


def exact_quantized(b, group, with_zeros):
    n, k = b.shape
    out = torch.empty(n, k, dtype=torch.float64, device=b.device)
    for i in range(0, n, group):
        block = b[i:i + group]
        if with_zeros:
            hi, lo = block.max(0).values.clamp(min=0), block.min(0).values.clamp(max=0)
            s = ((hi - lo) / 15).to(torch.bfloat16).double()
            z = torch.nan_to_num(torch.round(-lo / s)).clamp(0, 15)
            q = torch.nan_to_num(torch.round(block / s) + z).clamp(0, 15)
        else:
            s = (block.abs().max(0).values / 7).to(torch.bfloat16).double()
            z = 0.0
            q = torch.nan_to_num(torch.round(block / s)).clamp(-8, 7)
        out[i:i + group] = s * (q - z)
    return out


def exact_values(w, which):
    """s (q - z) in 64 bits, row by row from the group that the row is in."""
    codes = w["codes"][which]
    group_of = torch.arange(codes.shape[-2], device=codes.device) // w["group"]
    s = w["scales"][which].double().index_select(-2, group_of)
    if w["zeros"] is None:
        return s * (codes.double() - 8)
    return s * (codes.double() - w["zeros"][which].double().index_select(-2, group_of))


def exact_moe(case, gen, dtype):
    t, d, f, e, top = case["t"], case["d"], case["f"], case["e"], case["top"]
    x = activations(gen, t, d, dtype).double()
    live = torch.rand(t, generator=gen, device="cuda") < 0.7 if case["masked"] else None
    router = weights(gen, d, e, d).to(dtype).double()
    mats = [quantized(gen, case, (e,), n, k, torch.bfloat16) for n, k in ((d, f), (d, f), (f, d))]
    logits = (x @ router.T).cpu()
    y = torch.zeros(t, d, dtype=torch.float64, device=x.device)
    shares = torch.zeros(t, top, dtype=torch.float64)
    users = {}
    for row in range(t):
        if live is not None and not bool(live[row]):
            continue
        line = logits[row].tolist()
        chosen = sorted(sorted(range(e), key=lambda j: (-line[j], j))[:top])
        biggest = max(line)
        p = [math.exp(line[j] - biggest) for j in chosen]
        total = sum(p) if case["renorm"] else sum(math.exp(v - biggest) for v in line)
        for slot, j in enumerate(chosen):
            shares[row, slot] = p[slot] / total
            users.setdefault(j, []).append((row, p[slot] / total))
    for j, rows in sorted(users.items()):
        index = torch.tensor([r for r, _ in rows], device=x.device)
        share = torch.tensor([s for _, s in rows], dtype=torch.float64, device=x.device)
        gate, up, down = (exact_values(m, j) for m in mats)
        g = x[index] @ gate
        h = g / (1 + torch.exp(-g)) * (x[index] @ up)
        y.index_add_(0, index, (h @ down) * share[:, None])
    return y, None, shares.to(x.device)


# ---- what a pass cannot do without --------------------------------------------------

def weight_bytes(case, n, k):
    groups = -(-n // case["group"])
    return n * k / 2 + groups * k * (2.5 if case["zeros"] else 2)


def work(case):
    size = BYTES[case["dtype"]]
    if case["op"] == "quantize":
        n, k = case["n"], case["k"]
        # read the weights, write the codes, read them back, write the values
        return {"bytes": n * k * (size + 4) + 2 * weight_bytes(case, n, k), "flops": 2 * n * k}
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": weight_bytes(case, n, k) + size * (m * n + m * k), "flops": 2 * m * n * k}
    t, d, f, e, top = case["t"], case["d"], case["f"], case["e"], case["top"]
    lively = t * (0.7 if case["masked"] else 1.0)
    read = e * (1 - (1 - top / e) ** lively)  # experts that some token picks
    return {"bytes": read * (2 * weight_bytes(case, d, f) + weight_bytes(case, f, d))
            + size * (e * d + 2 * t * d) + 8 * t * top,
            "flops": lively * (top * 6 * d * f + 2 * e * d)}

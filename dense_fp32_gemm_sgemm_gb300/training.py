"""What a training step spends on matrix products beside its layers: the cross entropy of an
output head, with its gradients, and orthogonalised updates.

Like the rest of the binding this marshals arguments only; the definitions and the limits are
those of ``sgemm_cross_entropy`` and ``sgemm_orthogonalize`` in the C header. As everywhere in the
binding, results are not part of autograd's graph, also where inputs require gradients: a loss that
is to be differentiated needs cross_entropy_grad, whose gradients the caller passes on.

    loss, losses, lse = sg.cross_entropy(x, weight, target)             # x: T x D, weight: V x D
    loss, losses, lse, dx, dweight = sg.cross_entropy_grad(x, weight, target)
    update = sg.orthogonalize(gradient)                                 # M x N, or a stack of them
"""

from __future__ import annotations

import ctypes
import operator
import struct
from typing import NamedTuple

import torch

from . import lib
from .q4 import _cuda_tensor, _dtype_code, _launch, _result, _rows

# The coefficients of each step, chosen to raise small singular values fast: five steps bring
# those of a normalised matrix to between 0.7 and 1.2 or so.
ORTHOGONALIZE_COEFFICIENTS = (3.4445, -4.7750, 2.0315)


# sgemm_ce's fields in their order and native alignment (its bytes are packed in a fifth of the time
# that a ctypes structure takes)
_CE = struct.Struct("@PqPqPiiiiiPPPPPqPq")


class CrossEntropy(NamedTuple):
    """``loss``: the weighted sum of the tokens' losses (no dimensions); ``losses`` and ``lse``:
    each token's loss and logarithm of the sum of exponentials (T). All float32."""
    loss: torch.Tensor
    losses: torch.Tensor
    lse: torch.Tensor


class CrossEntropyGrad(NamedTuple):
    """As CrossEntropy, with the gradients of ``loss`` with respect to x and weight, in their
    type (None where not asked for)."""
    loss: torch.Tensor
    losses: torch.Tensor
    lse: torch.Tensor
    dx: torch.Tensor | None
    dweight: torch.Tensor | None


def _given_or_new(t, name, like, stream):
    """An output like ``like`` and its row pitch: the given tensor, checked, or a new one."""
    if t is None:
        return _result(like.shape, like.dtype, like.device, stream), like.shape[1]
    _cuda_tensor(t, name)
    if t.dtype != like.dtype or t.shape != like.shape or t.device != like.device:
        raise ValueError(f"{name} must be of shape {tuple(like.shape)} and type {like.dtype} on "
                         f"{like.device}")
    return t, _rows(t, name, like.shape[1])


def _cross_entropy(x, weight, target, token_weights, want_dx, want_dweight, dx, dweight, stream):
    _cuda_tensor(x, "x")
    _cuda_tensor(weight, "weight")
    _cuda_tensor(target, "target")
    code = _dtype_code(x, "x")
    if weight.dim() != 2 or 0 in weight.shape:
        raise ValueError(f"weight must be a V x D tensor, not {tuple(weight.shape)}")
    V, D = weight.shape
    if weight.dtype != x.dtype or weight.device != x.device:
        raise ValueError(f"weight is {weight.dtype} on {weight.device}, x {x.dtype} on {x.device}")
    ldx, ldw = _rows(x, "x", D), _rows(weight, "weight", D)
    T = x.shape[0]
    if target.dtype not in (torch.int64, torch.int32) or target.shape != (T,) or \
            not target.is_contiguous() or target.device != x.device:
        raise ValueError(f"target must be {T} int64 or int32 values on {x.device}")
    if token_weights is not None:
        _cuda_tensor(token_weights, "token_weights")
        if token_weights.dtype != torch.float32 or token_weights.shape != (T,) or \
                not token_weights.is_contiguous() or token_weights.device != x.device:
            raise ValueError(f"token_weights must be {T} float32 values on {x.device}")
    lddx = lddw = 0
    if want_dx:
        dx, lddx = _given_or_new(dx, "dx", x, stream)
    if want_dweight:
        dweight, lddw = _given_or_new(dweight, "dweight", weight, stream)
    loss = _result((), torch.float32, x.device, stream)
    losses = _result((T,), torch.float32, x.device, stream)
    lse = _result((T,), torch.float32, x.device, stream)
    if max(T, D, V) > 2 ** 31 - 1:
        raise ValueError(f"sizes of {T} x {D} by {V} are too large")
    args = _CE.pack(x.data_ptr(), ldx, weight.data_ptr(), ldw, target.data_ptr(),
                    64 if target.dtype is torch.int64 else 32, code, T, D, V,
                    0 if token_weights is None else token_weights.data_ptr(), loss.data_ptr(),
                    losses.data_ptr(), lse.data_ptr(), dx.data_ptr() if want_dx else 0, lddx,
                    dweight.data_ptr() if want_dweight else 0, lddw)
    _launch(lib().sgemm_cross_entropy, "sgemm_cross_entropy",
            (x, weight, target, token_weights, loss, losses, lse, dx, dweight),
            x.get_device(), stream, args)
    return loss, losses, lse, dx, dweight


def cross_entropy(x, weight, target, token_weights=None, stream=None) -> CrossEntropy:
    """Softmax cross entropy of the logits ``x @ weight.T``, which are not kept: x T x D, weight
    V x D (float32, bfloat16 or float16; rows may be slices of wider ones), target T integers.
    Tokens whose target is not in 0 .. V - 1 do not count; of them nothing is read.
    ``token_weights`` (T, float32): each token's share of ``loss``; without, one over the number
    of tokens that count. The results are values alone, without a graph for ``backward``."""
    return CrossEntropy(*_cross_entropy(x, weight, target, token_weights, False, False, None, None,
                                        stream)[:3])


def cross_entropy_grad(x, weight, target, token_weights=None, need_dx=True, need_dweight=True,
                       dx=None, dweight=None, stream=None) -> CrossEntropyGrad:
    """cross_entropy and the gradients of its ``loss`` with respect to x and weight, written to
    ``dx`` and ``dweight`` where they are given. With need_dx or need_dweight false that gradient
    is neither computed nor written. ``loss`` has no graph for ``backward``: the gradients are here."""
    for name, t, need in (("dx", dx, need_dx), ("dweight", dweight, need_dweight)):
        if t is not None and not need:
            raise ValueError(f"{name} is given but not needed")
    return CrossEntropyGrad(*_cross_entropy(x, weight, target, token_weights, need_dx, need_dweight,
                                            dx, dweight, stream))


def _layout(t, name):
    """(matrices, M, N, row pitch, stride) of a matrix or a stack of them."""
    if t.dim() not in (2, 3) or 0 in t.shape[-2:]:
        raise ValueError(f"{name} must be an M x N matrix or an E x M x N stack of them, not "
                         f"{tuple(t.shape)}")
    M, N = t.shape[-2:]
    pitch, step = t.stride()[-2:]
    if (N > 1 and step != 1) or (M > 1 and pitch < N):
        raise ValueError(f"{name} must have contiguous rows that do not overlap "
                         f"(strides {t.stride()})")
    pitch = pitch if M > 1 else max(pitch, N)
    count = t.shape[0] if t.dim() == 3 else 1
    stride = t.stride(0) if count > 1 else 0
    if count > 1 and stride < (M - 1) * pitch + N:
        raise ValueError(f"each of {name}'s matrices must begin behind the last element of the one "
                         f"before (strides {t.stride()})")
    return count, M, N, pitch, stride


def orthogonalize(G, steps: int = 5, coefficients=ORTHOGONALIZE_COEFFICIENTS, eps: float = 1e-7,
                  out=None, stream=None):
    """Newton-Schulz steps from G (M x N, or a stack E x M x N; float32, bfloat16 or float16)
    towards the nearest matrix with orthonormal rows (columns where M > N): X = G / (|G| + eps),
    then ``X = a X + (b A + c A A) X`` with ``A = X X^T`` for each step. ``coefficients``: a, b, c
    for all steps or a sequence of one such triple for each. ``out`` may be G itself."""
    steps = operator.index(steps)
    _cuda_tensor(G, "G")
    code = _dtype_code(G, "G")
    count, M, N, ldg, stride_g = _layout(G, "G")
    triples = [tuple(c) if isinstance(c, (tuple, list)) else c for c in coefficients]
    if triples and not isinstance(triples[0], tuple):
        triples = [tuple(triples)] * steps
    if steps < 1 or len(triples) != steps or any(not isinstance(c, tuple) or len(c) != 3
                                                 for c in triples):
        raise ValueError(f"coefficients must be three numbers, or three for each of {steps} steps "
                         "(at least one)")
    if out is None:
        out = _result(G.shape, G.dtype, G.device, stream)
    else:
        _cuda_tensor(out, "out")
        if out.dtype != G.dtype or out.shape != G.shape or out.device != G.device:
            raise ValueError(f"out must be of shape {tuple(G.shape)} and type {G.dtype} on "
                             f"{G.device}")
    _, _, _, ldo, stride_o = _layout(out, "out")
    flat = (ctypes.c_float * (3 * steps))(*(float(v) for c in triples for v in c))
    _launch(lib().sgemm_orthogonalize, "sgemm_orthogonalize", (G, out), G.get_device(), stream,
            G.data_ptr(), code, count, M, N, ldg, stride_g, out.data_ptr(), ldo, stride_o, steps,
            flat, float(eps))
    return out

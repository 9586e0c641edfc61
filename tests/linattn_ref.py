"""Linear attention with a per-head decay and layer norm in 64 bits, by their definitions, with the bounds that the
kernels' results are held to.

The reference runs the recurrence step by step in float64 (torch, CPU) and differentiates it by torch's autograd.
Bounds are proved element by element from the magnitude M of a result: the same quantity computed from the absolute
values of all inputs. With u = 2^-24 (fp32's half step), a result that sums at most n products in fp32, each operand
exact, is off by at most n·u·M. n counts, for every path from an input to the result: the widths of the products
(N + P), the steps of a chunk (64), and per chunk passed the state's scaling and adding (4); and the decays: e^d is
taken of a difference of sums rounded to fp32 and multiplied by log2 e, so it is off by (2|d| + 2)·u, summed over the
path 2·104 + 2 per chunk at most (past |d| = 104 e^d is below fp32's range, and the product is 0, an absolute error
below 2^-125 times the operands). bf16 adds, for results in bf16, the one rounding of the state or adjoint on a path
through it, or of the scores on a path through them (2^-8 of the product; a path takes one of the two), operands cut into
two parts (2^-16, at most two on a path), and the rounding of the result (2^-8 of it); fp32 results take their fp32
operands in three parts (2^-24).
"""
import math

import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def recur(q, k, v, g, scale, first=None, lengths=None):
    """o [b, L, H, P] and the state after each row's last step, in the inputs' (float64) precision; differentiable."""
    b, L, G, N = q.shape
    H, P = v.shape[2:]
    head = torch.arange(H) // (H // G)
    g = g.expand(b, L, H)
    S = torch.zeros(b, H, P, N, dtype=q.dtype) if first is None else first
    outs = []
    for t in range(L):
        live = torch.ones(b, dtype=torch.bool) if lengths is None else t < lengths.clamp(0, L)
        m = live[:, None, None, None]
        new = torch.exp(g[:, t])[..., None, None] * S + v[:, t][..., :, None] * k[:, t][:, head][..., None, :]
        S = torch.where(m, new, S)
        o = scale * (S * q[:, t][:, head][..., None, :]).sum(-1)
        outs.append(torch.where(m[..., 0], o, torch.zeros_like(o)))
    return (torch.stack(outs, 1) if outs else torch.zeros(b, 0, H, P, dtype=q.dtype)), S


def grads(q, k, v, g, scale, do, first=None, d_final=None, lengths=None):
    """Gradients of sum(do·o) + sum(d_final·state) by autograd through recur."""
    leaves = [t.detach().clone().requires_grad_() for t in (q, k, v, g)]
    init = None if first is None else first.detach().clone().requires_grad_()
    if init is None:
        b, H, P, N = v.shape[0], v.shape[2], v.shape[3], q.shape[3]
        init = torch.zeros(b, H, P, N, dtype=q.dtype).requires_grad_()
    o, S = recur(*leaves, scale, init, lengths)
    loss = (do * o).sum() + (0 if d_final is None else (d_final * S).sum()) + 0 * sum(t.sum() for t in leaves)
    got = torch.autograd.grad(loss, leaves + [init])
    return dict(zip(("dq", "dk", "dv", "dg", "d_initial_state"), got))


def paths(L, N, P, ratio=1):
    """n of the bound above."""
    return N + P + 64 + 6 * math.ceil(max(L, 1) / 64) + 210 + ratio


def bound(ref, mag, dtype, L, N, P, out_dtype=None, ratio=1):
    """How far a result may be from `ref`, element by element; dtype: of the inputs, out_dtype: of the result."""
    out_dtype = out_dtype or dtype
    parts = 2.0 ** -8 + 2 * 2.0 ** -16 if dtype == torch.bfloat16 and out_dtype == torch.bfloat16 else 0.0
    n = paths(L, N, P, ratio)
    return HALF[out_dtype] * ref.abs() + (parts + (n + 8) * U) * mag + 2.0 ** -110


def assert_within(got, ref, tol, what):
    got = got.detach().double().cpu()
    assert got.shape == ref.shape, f"{what}: shape {tuple(got.shape)}, expected {tuple(ref.shape)}"
    assert torch.isfinite(got).all(), f"{what}: non-finite values"
    over = (got - ref).abs() - tol
    if over.numel():
        i = int(over.argmax())
        at = tuple(int(x) for x in torch.unravel_index(torch.tensor(i), over.shape))
        assert over.flatten()[i] <= 0, (f"{what}: |{got[at]:.8g} - {ref[at]:.8g}| = {(got - ref).abs()[at]:.3e} > "
                                        f"{tol.expand_as(ref)[at]:.3e} at {at}")

"""Softmax attention, its gradient and the position rotation in 64 bits, by their definitions, with the bounds that the
kernels' results are held to.

Bounds, with u = 2^-24 (fp32's half step). A score is a sum of D products, exact (bf16) or rounded (fp32): it is off by at
most (D + 2)·u·a, a = scale·Σ|q_d k_d|, times log2 e and minus the maximum by two more roundings of numbers of at most 2a (a
score) and |lse| or a maximum of at most max a: a weight is off by e = (D + 8)·u·A relative to its value, A = max over the row of a and
|lse|, and by the exponential's own 2 roundings and 2 for each of the rescalings, of which there is at most one a tile of 32 keys:
e = (D + 8)·u·A + (2·tiles + 4)·u. A row's output is Σ p v / Σ p, each sum of n terms: off by (2e + (n + 4)·u)·Σ p|v|; with bf16
the weights enter rounded, 2^-8 of p|v| each, and the result is rounded. lse is off by e + (n + 4)·u + 4u·|lse|.

Gradients: delta = do·o is off by |do|·(what o is off by) + D·u·|do||o|, do·v by (D + 1)·u·Σ|do||v|, so ds = p(do·v − delta) by
p·(e'·(|do·v| + |delta|) + both), e' = e + 2u·|lse|. ds and p enter products rounded to bf16, 2^-8; sums over n terms of
magnitude t add n·u·Σt; the result is rounded.
"""
import math

import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
PART = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8}


def visible(nq, nk, causal):
    i, j = torch.arange(nq)[:, None], torch.arange(nk)[None, :]
    return j <= i + nk - nq if causal else torch.ones(nq, nk, dtype=torch.bool)


def one(q, k, v, scale, causal, see=None):
    """q [nq, H, D], k and v [nk, G, D] in float64 -> o [nq, H, D], lse [nq, H]; differentiable."""
    H, G = q.shape[1], k.shape[1]
    head = torch.arange(H) // (H // G)
    s = scale * torch.matmul(q.transpose(0, 1), k[:, head].permute(1, 2, 0))
    if see is None:
        see = visible(q.shape[0], k.shape[0], causal)
    s = torch.where(see, s, torch.full((), -math.inf, dtype=s.dtype))
    empty = ~see.any(-1)
    lse = torch.logsumexp(torch.where(empty[:, None], torch.zeros((), dtype=s.dtype), s), -1) if s.shape[-1] else \
        torch.zeros(H, q.shape[0], dtype=s.dtype)
    p = torch.where(see, torch.exp(s - lse[..., None]), torch.zeros((), dtype=s.dtype))
    o = torch.matmul(p, v[:, head].transpose(0, 1)).transpose(0, 1)
    lse = torch.where(empty, torch.full((), -math.inf, dtype=s.dtype), lse).t()
    return o, lse


def _weights(q, k, scale, lse, see):
    """p and the magnitudes a of the scores, [H, nq, nk]."""
    head = torch.arange(q.shape[1]) // (q.shape[1] // k.shape[1])
    dot = lambda x, y: torch.matmul(x.transpose(0, 1), y[:, head].permute(1, 2, 0))  # noqa: E731
    s, a = scale * dot(q, k), abs(scale) * dot(q.abs(), k.abs())
    p = torch.where(see, torch.exp(s - lse.t()[..., None].clamp_min(-1e300)), torch.zeros((), dtype=s.dtype))
    return p, torch.where(see, a, torch.zeros((), dtype=s.dtype)), head


def relative(a, lse, D, nk):
    """e of a row [H, nq, 1]."""
    if nk == 0:
        return torch.zeros(*a.shape[:2], 1, dtype=torch.float64)
    top = torch.maximum(a.amax(-1, keepdim=True), lse.t()[..., None].abs().nan_to_num(0, 0, 0))
    return (D + 8) * U * top + (2 * math.ceil(nk / 32) + 4) * U


def bounds(q, k, v, scale, causal, dtype, see=None):
    """How far o and lse of one sequence may be from one()'s."""
    see = visible(q.shape[0], k.shape[0], causal) if see is None else see
    o, lse = one(q, k, v, scale, causal, see)
    p, a, head = _weights(q, k, scale, lse, see)
    D, nk = q.shape[2], k.shape[0]
    e = relative(a, lse, D, nk)
    mag = torch.matmul(p, v[:, head].transpose(0, 1).abs())
    tol_o = ((2 * e + (nk + 4) * U + PART[dtype]) * mag).transpose(0, 1) + HALF[dtype] * o.abs() * 1.01 + 2.0 ** -110
    tol_lse = (e.squeeze(-1) + (nk + 4) * U).t() + 4 * U * lse.abs().nan_to_num(0, 0, 0)
    return o, lse, tol_o, tol_lse


def grads(q, k, v, do, scale, causal):
    leaves = [t.detach().clone().requires_grad_() for t in (q, k, v)]
    o, _ = one(*leaves, scale, causal)
    return torch.autograd.grad((o * do).sum() + 0 * sum(t.sum() for t in leaves), leaves)


def grad_bounds(q, k, v, do, scale, causal, dtype):
    """dq, dk, dv of one sequence and how far results may be from them."""
    see = visible(q.shape[0], k.shape[0], causal)
    o, lse, tol_o, _ = bounds(q, k, v, scale, causal, dtype)
    dq, dk, dv = grads(q, k, v, do, scale, causal)
    p, a, head = _weights(q, k, scale, lse, see)
    nq, H, D = q.shape
    nk, G = k.shape[:2]
    e = relative(a, lse, D, nk) + 2 * U * lse.t()[..., None].abs().nan_to_num(0, 0, 0)
    heads = lambda t: t.transpose(0, 1)  # noqa: E731
    dp = torch.matmul(heads(do), v[:, head].permute(1, 2, 0))
    off_dp = (D + 1) * U * torch.matmul(heads(do).abs(), v[:, head].abs().permute(1, 2, 0))
    delta = (do * o).sum(-1).t()[..., None]
    off_delta = ((do.abs() * (tol_o + D * U * o.abs())).sum(-1)).t()[..., None]
    ds = p * (dp - delta)
    off = p * (e * (dp.abs() + delta.abs()) + off_dp + off_delta + 2 * U * (dp.abs() + delta.abs()))
    part = PART[dtype]
    size = lambda n: part * 1.01 + (n + 4) * U  # noqa: E731
    t_q = abs(scale) * torch.matmul(off + size(nk) * (ds.abs() + off), k[:, head].transpose(0, 1).abs()).transpose(0, 1)
    wide_k = abs(scale) * torch.matmul((off + size(nq * H // G) * (ds.abs() + off)).transpose(1, 2), heads(q).abs())
    wide_v = torch.matmul((p * (e + size(nq * H // G))).transpose(1, 2), heads(do).abs())
    fold = lambda t: t.reshape(G, H // G, nk, D).sum(1).transpose(0, 1)  # noqa: E731
    end = lambda t, ref: t + HALF[dtype] * (ref.abs() + t) + 2.0 ** -110  # noqa: E731
    return (dq, dk, dv), (end(t_q, dq), end(fold(wide_k), dk), end(fold(wide_v), dv))


def rotate(x, pos, freq, interleaved, inverse=False):
    """x [T, heads, D] float64 turned at positions pos [T]; and the magnitude of each result's two terms."""
    R = 2 * freq.numel()
    angle = pos.double()[:, None, None] * freq * (-1 if inverse else 1)
    c, s = torch.cos(angle), torch.sin(angle)
    one_, two = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    y, m = x.clone(), x.abs()
    a, b = x[..., one_], x[..., two]
    y[..., one_], y[..., two] = a * c - b * s, b * c + a * s
    m[..., one_] = m[..., two] = a.abs() + b.abs()
    return y, m


def rotation_bound(y, m, dtype):
    """Angles are reduced in 64 bits to a fraction of a turn, rounded to fp32 (2^-25·2π), sine and cosine taken to 2 units of
    2^-23, and two products added with one rounding each."""
    return HALF[dtype] * y.abs() * 1.01 + (2.0 ** -25 * 2 * math.pi + 4 * U + 3 * U) * m


def assert_within(got, ref, tol, what):
    got, ref = got.detach().double().cpu(), ref.double()
    assert got.shape == ref.shape, f"{what}: shape {tuple(got.shape)}, expected {tuple(ref.shape)}"
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinite values differ"
    assert torch.isfinite(got[~inf]).all(), f"{what}: non-finite values"
    over = torch.where(inf, torch.zeros((), dtype=ref.dtype), (got - ref).abs() - tol)
    if over.numel():
        i = int(over.nan_to_num(math.inf).argmax())
        at = tuple(int(x) for x in torch.unravel_index(torch.tensor(i), over.shape))
        assert over.flatten()[i] <= 0, (f"{what}: |{got[at]:.8g} - {ref[at]:.8g}| = {(got - ref).abs()[at]:.3e} > "
                                        f"{tol.expand_as(ref)[at]:.3e} at {at}")

"""How exactly softmax attention computes with bf16: results are the definition's but for their own rounding and what fp32 sums leave.

The bounds are those of softmax_ref.py but that weights enter products in two bf16 parts, the second of which is what the first
leaves, rounded: (2^-8)^2 = 2^-16 of each instead of 2^-8. Results of one part are outside of them wherever a sum's terms cancel
(test_one_part_is_outside shows it on the CPU).

delta, as the gradient's kernels form it with D' = do·o of a rounded o: D' + Σ_j p_j (do·v_j − D'). Weights off by e of their value
(their sum so off 1 by e), products by (D + 1)·u·(Σ|do||v_j| + |D'|), and a sum of nk terms make of that
Σ_j p_j ((e + (nk + 4)·u)(|do·v_j| + |D'|) + (D + 1)·u·(Σ|do||v_j| + |D'|)) + 4u·|D'|, where |D'| <= |delta| + Σ|do|·(what o is off by).
Where what is left could be more than 2^-7·Σ|do o|, the kernels take D' itself (grad_bounds).

Norms: rounding alone puts a result ‖x − bf16(x)‖ off, 1.6e-3 of its norm. 1.1 of that leaves 0.45 of it, 7e-4, to all else, which is
independent of it: two parts (2^-16 = 1.5e-5 of each weight) and fp32 products (below 1e-4 for these sizes, keys of 4 deviations'
offset among them). One part of ds or of the weights (1.2 to 1.4 of that) or a delta from the rounded o (1.2, with
offsets of the keys up to 6) does not fit in."""
import math

import pytest
import torch

import softmax_ref as R
from selective_state_space_82_amd import api

F32, BF16 = torch.float32, torch.bfloat16
PARTS = 2.0 ** -16
gpu = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _two_parts(monkeypatch):
    monkeypatch.setitem(R.PART, BF16, PARTS)


@pytest.fixture
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no ROCm GPU visible")
    return api.lib()


def normal(seed, *shapes, shift=0.0):
    """bf16 values on the CPU, in float64; the second (the keys) share an offset of `shift` in every coordinate."""
    r = torch.Generator().manual_seed(seed)
    return [(torch.randn(s, generator=r) + (shift if i == 1 else 0.0)).bfloat16().double() for i, s in enumerate(shapes)]


def test_one_part_is_outside():
    """Weights rounded to bf16 once, all else exact."""
    q, k, v = normal(0, (200, 2, 64), (200, 2, 64), (200, 2, 64))
    o, lse, tol, _ = R.bounds(q, k, v, 0.125, True, BF16)
    p, _, _ = R._weights(q, k, 0.125, lse, R.visible(200, 200, True))
    one = torch.matmul(p.bfloat16().double(), v.transpose(0, 1)).transpose(0, 1)
    hi = p.bfloat16().double()
    two = torch.matmul(hi + (p - hi).bfloat16().double(), v.transpose(0, 1)).transpose(0, 1)
    assert ((one.bfloat16().double() - o).abs() > tol).double().mean() > 0.05
    assert ((two.bfloat16().double() - o).abs() <= tol).all()


# whole walks; one cut into pieces; tiles of 96 columns and a view's element-wise path
FORWARD = [(300, 300, 4, 2, 64, False), (1500, 1500, 2, 1, 128, False), (90, 700, 2, 2, 80, False), (300, 300, 2, 1, 128, True)]


@gpu
@pytest.mark.parametrize("nq,nk,H,G,D,odd", FORWARD)
@pytest.mark.parametrize("causal", [True, False])
def test_prompt(lib, nq, nk, H, G, D, odd, causal):
    q, k, v = normal(D, (nq, H, D), (nk, G, D), (nk, G, D))
    ref, lse, tol, _ = R.bounds(q, k, v, D ** -0.5, causal, BF16)
    t = [x.bfloat16()[None].cuda() for x in (q, k, v)]
    if odd:  # keys at an odd offset
        wide = torch.empty(1, nk, G * D + 1, dtype=BF16, device="cuda")
        t[1] = wide[..., 1:].unflatten(-1, (G, D)).copy_(t[1])
    R.assert_within(api.ssm_attn_fwd(*t, causal=causal)[0], ref, tol, "o")


@gpu
def test_prompt_with_a_nan_behind_it(lib):
    """A block that is done again for a NaN in a masked place."""
    q, k, v = normal(5, (300, 2, 64), (300, 1, 64), (300, 1, 64))
    ref, _, tol, _ = R.bounds(q, k, v, 0.125, True, BF16)
    v[290, 0, 3] = math.nan
    o = api.ssm_attn_fwd(*(x.bfloat16()[None].cuda() for x in (q, k, v)))[0]
    R.assert_within(o[:290], ref[:290], tol[:290], "o")


@gpu
@pytest.mark.parametrize("H,G,D,page,lens", [(4, 2, 64, 16, [200, 1, 63]), (40, 2, 128, 64, [250]), (2, 1, 96, 7, [3000, 40]),
                                             (3, 3, 30, 5, [90])])
def test_one_token(lib, H, G, D, page, lens):
    b, most = len(lens), -(-max(lens) // page)
    q, kc, vc = normal(D, (b, H, D), (b * most, page, G, D), (b * most, page, G, D))
    table = torch.arange(b * most).flip(0).view(b, most)
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    o = api.ssm_attn_step(*(x.bfloat16().cuda() for x in (q, kc, vc)), table.int().cuda(), n)
    for i, m in enumerate(lens):
        k, v = (c[table[i]].flatten(0, 1)[:m] for c in (kc, vc))
        ref, _, tol, _ = R.bounds(q[i:i + 1], k, v, D ** -0.5, True, BF16)
        R.assert_within(o[i:i + 1], ref, tol, f"row {i}")


# whole walks; walks cut into pieces; 96 columns; rows without 16-byte accesses; more keys than queries
GRADIENT = [(2000, 2000, 24, 24, 64), (300, 300, 4, 2, 128), (1500, 1500, 2, 1, 64), (133, 133, 6, 2, 96), (130, 300, 2, 2, 30)]


def gradients(nq, nk, H, G, D, causal, shift=0.0):
    q, k, v, do = normal(D + nq, (nq, H, D), (nk, G, D), (nk, G, D), (nq, H, D), shift=shift)
    t = [x.bfloat16()[None].cuda() for x in (q, k, v, do)]
    o, lse = api.ssm_attn_fwd(*t[:3], causal=causal, return_lse=True)
    g = api.ssm_attn_bwd(*t[:3], o=o, lse=lse, do=t[3], causal=causal)
    return (q, k, v, do), {n: x[0] for n, x in g.items()}


def grad_bounds(q, k, v, do, scale, causal, given=None):
    """dq, dk, dv of one sequence and how far results may be from them. given: (o, lse) of more keys than these, whose delta do·o
    is then taken as it is."""
    nq, H, D = q.shape
    nk, G = k.shape[:2]
    see = R.visible(nq, nk, causal)
    o, lse, tol_o, _ = R.bounds(q, k, v, scale, causal, BF16)
    if given is not None:
        o, lse, tol_o = given
    p, a, head = R._weights(q, k, scale, lse, see)
    first = lambda t: t.transpose(0, 1)  # noqa: E731  heads first
    e = R.relative(a, lse, D, nk) + 2 * R.U * lse.t()[..., None].abs().nan_to_num(0, 0, 0)
    dp = torch.matmul(first(do), v[:, head].permute(1, 2, 0))
    size_dp = torch.matmul(first(do).abs(), v[:, head].abs().permute(1, 2, 0))
    delta = (do * o).sum(-1).t()[..., None]
    of_o = (do.abs() * tol_o).sum(-1).t()[..., None]
    rough = of_o + D * R.U * (do.abs() * o.abs()).sum(-1).t()[..., None]
    d0 = delta.abs() + rough
    off_dp = (D + 1) * R.U * (size_dp + d0)
    fine = (p * ((e + (nk + 4) * R.U) * (dp.abs() + d0) + off_dp)).sum(-1, keepdim=True) + 4 * R.U * d0
    surely = rough + fine < 2.0 ** -7 * (1 - 2.0 ** -7) * (do.abs() * o.abs()).sum(-1).t()[..., None]
    off_delta = torch.where(surely, fine, torch.maximum(fine, rough)) if given is None else rough
    ds = p * (dp - delta)
    off = p * (e * (dp.abs() + delta.abs()) + off_dp + off_delta + 2 * R.U * (dp.abs() + delta.abs()))
    size = lambda n: R.PART[BF16] * 1.01 + (n + 4) * R.U  # noqa: E731
    dq = scale * torch.matmul(ds, first(k[:, head])).transpose(0, 1)
    dk = scale * torch.matmul(ds.transpose(1, 2), first(q))
    dv = torch.matmul(p.transpose(1, 2), first(do))
    t_q = abs(scale) * torch.matmul(off + size(nk) * (ds.abs() + off), first(k[:, head]).abs()).transpose(0, 1)
    t_k = abs(scale) * torch.matmul((off + size(nq * H // G) * (ds.abs() + off)).transpose(1, 2), first(q).abs())
    t_v = torch.matmul((p * (e + size(nq * H // G))).transpose(1, 2), first(do).abs())
    fold = lambda t: t.reshape(G, H // G, nk, D).sum(1).transpose(0, 1)  # noqa: E731
    end = lambda t, ref: t + R.HALF[BF16] * (ref.abs() + t) + 2.0 ** -110  # noqa: E731
    dk, dv = fold(dk), fold(dv)
    return (dq, dk, dv), (end(t_q, dq), end(fold(t_k), dk), end(fold(t_v), dv))


def test_the_bounds_are_of_the_same_gradient():
    x = normal(0, (40, 4, 16), (60, 2, 16), (60, 2, 16), (40, 4, 16))
    for a, b in zip(grad_bounds(*x, 0.25, True)[0], R.grads(*x, 0.25, True)):
        assert (a - b).abs().max() <= 1e-12 * b.abs().max()


def norms(g, ref):
    for n, want in zip(("dq", "dk", "dv"), ref):
        own = (want - want.bfloat16().double()).norm()
        off = (g[n].double().cpu() - want).norm()
        assert off <= 1.1 * own, f"{n}: {off / own:.3f} of its own rounding ({own / want.norm():.2e})"


@gpu
@pytest.mark.parametrize("nq,nk,H,G,D", GRADIENT)
@pytest.mark.parametrize("causal", [True, False])
def test_gradient(lib, nq, nk, H, G, D, causal):
    x, g = gradients(nq, nk, H, G, D, causal)
    few = [t[:, : t.shape[1] // G] for t in x]  # the first key head and its queries' heads
    got = {n: t[:, : t.shape[1] // G] for n, t in g.items()}
    ref, tol = grad_bounds(*few, D ** -0.5, causal)
    for n, r, t in zip(("dv", "dk", "dq"), ref[::-1], tol[::-1]):
        R.assert_within(got[n], r, t, n)
    norms(got, ref)


@gpu
@pytest.mark.parametrize("shift", [1.0, 4.0])
@pytest.mark.parametrize("L,H,G,D", [(64, 2, 2, 64), (512, 4, 2, 64), (1500, 2, 1, 128), (2000, 24, 24, 64)])
def test_keys_that_share_an_offset(lib, L, H, G, D, shift):
    """dq does not change with what all keys have in common, and its error does not grow with it."""
    x, g = gradients(L, L, H, G, D, True, shift)
    ref, _ = grad_bounds(*(t[:, : t.shape[1] // G] for t in x), D ** -0.5, True)
    norms({n: t[:, : t.shape[1] // G] for n, t in g.items()}, ref)


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("L,cut", [(300, 170), (1500, 64)])
def test_keys_in_shards(lib, L, cut, dtype):
    """o and lse of all keys, the gradient of some of them in each call: dk and dv are theirs, and dq adds up."""
    q, k, v, do = normal(L, (L, 2, 64), (L, 1, 64), (L, 1, 64), (L, 2, 64))
    t = [x.to(dtype)[None].cuda() for x in (q, k, v, do)]
    o, lse = api.ssm_attn_fwd(*t[:3], causal=False, return_lse=True)
    whole = R.bounds(q, k, v, 0.125, False, BF16)
    dq, tol_q = 0.0, 0.0
    got_q = torch.zeros(L, 2, 64, dtype=torch.float64)
    for part in (slice(0, cut), slice(cut, L)):
        g = api.ssm_attn_bwd(t[0], t[1][:, part], t[2][:, part], o=o, lse=lse, do=t[3], causal=False)
        ref, tol = grad_bounds(q, k[part], v[part], do, 0.125, False, given=whole[:3])
        for n, r, e in zip(("dv", "dk"), ref[:0:-1], tol[:0:-1]):
            R.assert_within(g[n][0], r, e, n)
        R.assert_within(g["dq"][0], ref[0], tol[0], "dq")
        got_q += g["dq"][0].double().cpu()
        dq, tol_q = dq + ref[0], tol_q + tol[0]
    assert ((got_q - dq).abs() <= tol_q).all()
    full = R.grads(q, k, v, do, 0.125, False)[0]
    assert (dq - full).abs().max() <= 1e-12 * full.abs().max()

"""Softmax attention over prompts and its gradient on the GPU (ssm_attn_fwd, ssm_attn_bwd) against their definitions in
64 bits (softmax_ref.py, which derives the bounds)."""
import math

import pytest
import torch

import softmax_ref as R
from selective_state_space_82_amd import api

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no ROCm GPU visible")
    api.lib()


def make(lens, H, G, D, dtype=F32, lens_k=None, layout="packed", seed=0, std=1.0):
    """Inputs on the CPU; every value is exact in `dtype`. rows: of each sequence in the queries and in the keys."""
    r = torch.Generator().manual_seed(seed)
    n = lambda *s: (std * torch.randn(s, generator=r)).to(dtype)  # noqa: E731
    lens_k = lens if lens_k is None else lens_k
    x = {"lens": lens, "lens_k": lens_k, "layout": layout}
    if layout == "packed":
        lead, lead_k = (sum(lens) + 3,), (sum(lens_k) + 2,)  # tokens of no sequence behind the last
    else:
        lead, lead_k = (len(lens), max(lens)), (len(lens), max(lens_k))
    x["q"], x["k"], x["v"], x["do"] = n(*lead, H, D), n(*lead_k, G, D), n(*lead_k, G, D), n(*lead, H, D)
    return x


def spans(x):
    """(rows of the queries, rows of the keys) of every sequence."""
    out, a, b = [], 0, 0
    for i, (n, m) in enumerate(zip(x["lens"], x["lens_k"])):
        out.append((slice(a, a + n), slice(b, b + m)) if x["layout"] == "packed" else ((i, slice(0, n)), (i, slice(0, m))))
        a, b = a + n, b + m
    return out


def where(x):
    i32 = dict(dtype=torch.int32, device="cuda")
    if x["layout"] == "packed":
        cu = lambda lens: torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)  # noqa: E731
        kw = dict(cu_seqlens=cu(x["lens"]), max_len=max(x["lens"]))
        if x["lens_k"] != x["lens"]:
            kw.update(cu_seqlens_k=cu(x["lens_k"]), max_len_k=max(x["lens_k"]))
        return kw
    if x["layout"] == "padded":
        return dict(lengths=torch.tensor(x["lens"], **i32), lengths_k=torch.tensor(x["lens_k"], **i32))
    return {}


def expected(x, causal, scale, dtype, gradient):
    names = ("dq", "dk", "dv") if gradient else ("o", "lse")
    shape = {"o": x["q"].shape, "lse": x["q"].shape[:-1], "dq": x["q"].shape, "dk": x["k"].shape, "dv": x["v"].shape}
    ref = {n: torch.full(shape[n], -math.inf if n == "lse" else 0.0, dtype=torch.float64) for n in names}
    tol = {n: torch.zeros(shape[n], dtype=torch.float64) for n in names}
    for rq, rk in spans(x):
        q, k, v, do = (x[n][r].double() for n, r in (("q", rq), ("k", rk), ("v", rk), ("do", rq)))
        if gradient:
            got = R.grad_bounds(q, k, v, do, scale, causal, dtype)
            values, tols = got
        else:
            o, lse, to, tl = R.bounds(q, k, v, scale, causal, dtype)
            values, tols = (o, lse), (to, tl)
        for n, val, t in zip(names, values, tols):
            r = rk if n in ("dk", "dv") else rq
            ref[n][r], tol[n][r] = val, t
    return ref, tol


def check(x, causal=True, scale=None, gradient=True, view=lambda n, t: t, what=""):
    dtype, D = x["q"].dtype, x["q"].shape[-1]
    scale = D ** -0.5 if scale is None else scale
    t = {n: view(n, x[n].cuda()) for n in ("q", "k", "v", "do")}
    kw = dict(scale=scale, causal=causal, **where(x))
    o, lse = api.ssm_attn_fwd(t["q"], t["k"], t["v"], return_lse=True, **kw)
    torch.cuda.synchronize()
    ref, tol = expected(x, causal, scale, dtype, False)
    R.assert_within(o, ref["o"], tol["o"], what + " o")
    R.assert_within(lse, ref["lse"], tol["lse"], what + " lse")
    if not gradient:
        return
    g = api.ssm_attn_bwd(t["q"], t["k"], t["v"], o=o, lse=lse, do=t["do"], **kw)
    torch.cuda.synchronize()
    ref, tol = expected(x, causal, scale, dtype, True)
    for n in ("dv", "dk", "dq"):
        R.assert_within(g[n], ref[n], tol[n], f"{what} {n}")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("L", [1, 2, 31, 32, 33, 64, 65, 127, 128, 129, 257])
def test_lengths(L, dtype):
    check(make([L, L], 2, 2, 64, dtype, layout="rows", seed=L))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [1, 7, 8, 13, 16, 31, 32, 40, 64, 72, 80, 96, 100, 120, 127, 128])
def test_widths(D, dtype):
    check(make([70, 133], 2, 1, D, dtype, seed=D))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,G", [(1, 1), (3, 3), (6, 2), (8, 1), (40, 2)])
def test_heads(H, G, causal, dtype):
    check(make([150], H, G, 32, dtype, layout="rows", seed=H), causal)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("layout", ["packed", "padded"])
@pytest.mark.parametrize("lens", [[1], [5, 1, 0, 200, 64], [0, 3], [128, 256, 1], [17] * 9])
def test_sequences(lens, layout, causal, dtype):
    check(make(lens, 4, 2, 64, dtype, layout=layout, seed=sum(lens)), causal)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("layout", ["packed", "padded"])
def test_more_keys_or_queries(layout, causal, dtype):
    """Keys of earlier tokens; more queries than keys (the first see none); no keys at all."""
    check(make([1, 40, 130, 90, 5], 2, 1, 64, dtype, [77, 140, 130, 20, 0], layout, 5), causal)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("layout", ["packed", "padded"])
@pytest.mark.parametrize("lens,lens_k,H,G,D", [([1000, 300, 40], None, 2, 1, 64), ([700], [1500], 4, 1, 20),
                                               ([5, 900], [600, 300], 3, 3, 128), ([1, 2], [513, 1100], 1, 1, 33)])
def test_cut_walks(lens, lens_k, H, G, D, layout, causal, dtype):
    """Few blocks and long walks: cut into pieces that a second launch joins; pieces that some queries see nothing of."""
    check(make(lens, H, G, D, dtype, lens_k, layout, seed=D), causal)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0, 3.0])
def test_scales(scale, dtype):
    check(make([100], 2, 2, 32, dtype, layout="rows", seed=3), scale=scale)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_large_scores(dtype):
    """Scores of some hundreds: the running maximum moves often, most weights vanish."""
    check(make([300], 2, 1, 64, dtype, layout="rows", std=6.0, seed=9), gradient=False)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [24, 128, 30])
def test_views(dtype, D):
    """Slices of a packed projection, heads apart, and a broadcast gradient."""
    def view(n, t):
        if n == "do":
            return t
        buf = torch.randn(*t.shape[:-2], 3, t.shape[-2] + 1, D, device="cuda").to(t.dtype)
        s = buf[..., 1, 1:, :]
        s.copy_(t)
        return s
    check(make([70, 33], 4, 2, D, dtype, seed=D), view=view)
    x = make([70, 33], 4, 2, D, dtype, seed=D)
    x["do"] = x["do"][:1, :1].expand_as(x["do"])
    check(x, view=lambda n, t: t[:1, :1].expand_as(t) if n == "do" else t)
    y = make([65], 4, 2, D, dtype, layout="rows", seed=D)
    y["k"] = y["k"][:, :1].expand_as(y["k"])
    check(y, view=lambda n, t: t[:, :1].expand_as(t) if n == "k" else t, gradient=False)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_given_output_keeps_other_tokens(dtype):
    x = make([40, 20], 2, 1, 32, dtype)
    o = torch.full(x["q"].shape, 7.0, device="cuda", dtype=dtype)
    api.ssm_attn_fwd(x["q"].cuda(), x["k"].cuda(), x["v"].cuda(), o=o, **where(x))
    assert (o[60:] == 7).all() and not (o[:60] == 7).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [32, 128])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("name", ["k", "v"])
def test_not_finite_where_masked(name, bad, D, dtype):
    """A NaN or Inf in a key or value reaches the queries that see it, and no others; other sequences never."""
    x = make([150, 90], 2, 1, D, dtype, seed=1)
    clean = api.ssm_attn_fwd(x["q"].cuda(), x["k"].cuda(), x["v"].cuda(), **where(x)).cpu()
    t = x[name].clone()
    t[70, 0, 3] = bad
    x[name] = t
    o = api.ssm_attn_fwd(x["q"].cuda(), x["k"].cuda(), x["v"].cuda(), **where(x)).cpu()
    assert torch.equal(o[:70], clean[:70]) and torch.equal(o[150:], clean[150:])
    hit = ~torch.isfinite(o[70:150]) if name == "v" else torch.ones(0, dtype=torch.bool)
    if name == "v":
        assert hit[..., 3].all() and not hit[..., :3].any() and not hit[..., 4:].any()
    elif not math.isinf(bad):
        assert torch.isnan(o[70:150]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("at", [3, 700, 895])
def test_not_finite_in_a_cut_walk(at, dtype):
    x = make([900], 2, 1, 64, dtype, seed=1)
    run = lambda: api.ssm_attn_fwd(x["q"].cuda(), x["k"].cuda(), x["v"].cuda(), **where(x)).cpu()  # noqa: E731
    clean = run()
    x["v"] = x["v"].clone()
    x["v"][at, 0, 5] = math.nan
    o = run()
    assert torch.equal(o[:at], clean[:at]) and torch.isnan(o[at:900, :, 5]).all()
    assert torch.isfinite(o[..., :5]).all() and torch.isfinite(o[..., 6:]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_tokens_that_do_not_count(dtype):
    """NaN past the lengths of a padded batch and behind the last sequence: as if it were not there."""
    for layout in ("padded", "packed"):
        x = make([50, 90, 0], 4, 2, 64, dtype, layout=layout, seed=2)
        nan = {n: torch.full_like(x[n], math.nan) for n in ("q", "k", "v", "do")}
        for rq, rk in spans(x):
            for n, r in (("q", rq), ("k", rk), ("v", rk), ("do", rq)):
                nan[n][r] = x[n][r]
        x.update(nan)
        x_ref = {**x, **{n: x[n].nan_to_num(0.0) for n in nan}}
        ref, tol = expected(x_ref, True, 0.125, dtype, True)
        t = {n: x[n].cuda() for n in nan}
        kw = dict(scale=0.125, **where(x))
        o, lse = api.ssm_attn_fwd(t["q"], t["k"], t["v"], return_lse=True, **kw)
        assert torch.isfinite(o).all() and not torch.isnan(lse).any()
        if layout == "padded":
            junk = torch.arange(90, device="cuda")[None] >= torch.tensor(x["lens"], device="cuda")[:, None]
            o[junk], lse[junk] = math.nan, math.nan
        g = api.ssm_attn_bwd(t["q"], t["k"], t["v"], o=o, lse=lse, do=t["do"], **kw)
        for n in ("dv", "dk", "dq"):
            R.assert_within(g[n], ref[n], tol[n], f"{layout} {n}")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("name", ["q", "k", "v", "do"])
def test_not_finite_in_gradients(name, dtype):
    """A NaN in one token's inputs leaves the gradients of other sequences, and of tokens 128 away that do not see it, as
    they are."""
    x = make([700, 90], 2, 1, 64, dtype, seed=1)
    t = {n: x[n].cuda() for n in ("q", "k", "v", "do")}
    o, lse = api.ssm_attn_fwd(t["q"], t["k"], t["v"], return_lse=True, **where(x))
    run = lambda: api.ssm_attn_bwd(t["q"], t["k"], t["v"], o=o, lse=lse, do=t["do"], **where(x))  # noqa: E731
    clean = run()
    t[name] = t[name].clone()
    t[name][300, 0, 7] = math.nan
    got = run()
    for n in ("dq", "dk", "dv"):
        assert torch.equal(got[n][700:], clean[n][700:]), n
    if name in ("q", "do"):  # query 300: keys after it do not enter
        assert torch.equal(got["dq"][:300 - 127], clean["dq"][:300 - 127]) and torch.equal(got["dq"][428:700], clean["dq"][428:700])
        assert all(torch.equal(got[n][428:700], clean[n][428:700]) for n in ("dk", "dv"))
    else:  # key 300: queries before it do not see it
        assert torch.equal(got["dq"][:300 - 127], clean["dq"][:300 - 127])


def test_gradient_against_differences():
    """(f(x + h d) − f(x − h d)) / 2h in 64 bits of the forward's definition, against the kernel's gradient along d."""
    x = make([37, 20], 4, 2, 16, F32, seed=4)
    t = {n: x[n].cuda() for n in ("q", "k", "v", "do")}
    kw = dict(scale=0.3, **where(x))
    o, lse = api.ssm_attn_fwd(t["q"], t["k"], t["v"], return_lse=True, **kw)
    g = api.ssm_attn_bwd(t["q"], t["k"], t["v"], o=o, lse=lse, do=t["do"], **kw)
    r = torch.Generator().manual_seed(1)
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv")):
        d = torch.randn(x[name].shape, generator=r, dtype=torch.float64)

        def f(h):
            y = {n: x[n].double() for n in ("q", "k", "v")}
            y[name] = y[name] + h * d
            return sum((R.one(y["q"][a], y["k"][b], y["v"][b], 0.3, True)[0] * x["do"][a].double()).sum() for a, b in spans(x))

        h = 1e-4
        slope = float((f(h) - f(-h)) / (2 * h))
        got = float((g[grad].double().cpu() * d).sum())
        size = float((g[grad].double().cpu() * d).abs().sum())
        assert abs(got - slope) <= 1e-5 * size + 1e-6, (name, got, slope)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_same_results_again_alone_and_in_a_batch(dtype):
    x = make([130, 61, 200], 4, 2, 64, dtype, seed=6)
    t = {n: x[n].cuda() for n in ("q", "k", "v", "do")}
    kw = where(x)

    def both(t, kw):
        o, lse = api.ssm_attn_fwd(t["q"], t["k"], t["v"], return_lse=True, **kw)
        return [o, lse, *api.ssm_attn_bwd(t["q"], t["k"], t["v"], o=o, lse=lse, do=t["do"], **kw).values()]

    a, b = both(t, kw), both(t, kw)
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    cut = {n: v[130:191] for n, v in t.items()}
    alone = both(cut, dict(cu_seqlens=torch.tensor([0, 61], dtype=torch.int32, device="cuda"), max_len=61))
    assert all(torch.equal(u[130:191], v) for u, v in zip(a, alone))


def test_bad_offsets_stay_inside():
    """Offsets outside of the tokens, falling ones, and sequences longer than max_len: cut, never out of range."""
    x = make([64, 64], 2, 1, 32, F32)
    t = {n: x[n].cuda() for n in ("q", "k", "v", "do")}
    for cu, most in (([-5, 64, 1000], 200), ([64, 10, 128], 128), ([0, 128, 128], 40)):
        kw = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), max_len=most)
        o, lse = api.ssm_attn_fwd(t["q"], t["k"], t["v"], return_lse=True, **kw)
        g = api.ssm_attn_bwd(t["q"], t["k"], t["v"], o=o, lse=lse, do=t["do"], **kw)
        torch.cuda.synchronize()
        assert torch.isfinite(o).all() and all(torch.isfinite(v).all() for v in g.values())
    keep = torch.arange(t["q"].shape[0], device="cuda") < 40
    assert (o[~keep] == 0).all() and (o[keep] != 0).any()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_captured_and_replayed(dtype):
    x = make([130, 61], 4, 2, 64, dtype, seed=8)
    t = {n: x[n].cuda() for n in ("q", "k", "v", "do")}
    kw = where(x)

    def step():
        o, lse = api.ssm_attn_fwd(t["q"], t["k"], t["v"], return_lse=True, **kw)
        return [o, lse, *api.ssm_attn_bwd(t["q"], t["k"], t["v"], o=o, lse=lse, do=t["do"], **kw).values()]

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(3):
        y = make([130, 61], 4, 2, 64, dtype, seed=20 + seed)
        for n in t:
            t[n].copy_(y[n])
        graph.replay()
        torch.cuda.synchronize()
        got = [u.clone() for u in out]
        assert all(torch.equal(u, v) for u, v in zip(got, step()))


def test_on_another_stream():
    x = make([130, 61], 4, 2, 64, BF16, seed=8)
    t = {n: x[n].cuda() for n in ("q", "k", "v")}
    kw = where(x)
    want = api.ssm_attn_fwd(t["q"], t["k"], t["v"], **kw)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(api.ssm_attn_fwd(t["q"], t["k"], t["v"], **kw))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)

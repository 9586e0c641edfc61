"""The largest calls of linear attention and layer norm: HIP takes fewer than 2^32 threads to a launch, so what would need
more is refused before anything is launched, and what is just below runs."""
import ctypes

import pytest
import torch

from selective_state_space_82_amd import api
from test_attn_abi_host import SHAPE, bwd, fwd, norm_bwd, norm_fwd, step

I64 = ctypes.c_int64


def workspace(gradient, b, L, H, G, N, P, dtype=0):
    return api.lib().ssm_linattn_workspace(gradient, b, L, H, G, N, P, dtype, 1, ctypes.byref(I64()))


def test_linear_attention_launches():
    one = dict(G=1, N=4, P=4, L=1)
    assert fwd(b=1 << 17, H=64, **one) == SHAPE             # 2^23 workgroups of 512 threads
    assert workspace(0, 1 << 17, 1, 64, 1, 4, 4) == SHAPE
    assert workspace(0, (1 << 17) - 1, 1, 64, 1, 4, 4) == 0
    assert workspace(0, 1 << 16, 1, 64, 1, 4, 65) == SHAPE  # two blocks of value columns each
    assert workspace(0, (1 << 16) - 1, 1, 64, 1, 4, 65) == 0
    assert step(b=1 << 18, H=64, G=1, N=1, P=1) == SHAPE    # 2^24 workgroups of 256
    assert step(b=1 << 16, H=64, G=1, N=1, P=193) == SHAPE
    for L, b, P in ((1, 1 << 18, 4), (4097, 2048, 4), (4097, 1024, 128)):  # states and adjoints of every chunk
        assert bwd(b=b, H=64, G=1, N=4, P=P, L=L) == SHAPE
        assert workspace(1, b, L, 64, 1, 4, P) == SHAPE
    assert workspace(1, 2016, 4097, 64, 1, 4, 4) == 0       # 64 · 2016 rows of 65 chunks: 129 walks each, below 2^24
    assert workspace(1, 2 ** 14, 1, 64, 1, 128, 64) == SHAPE  # 2^33 state elements: 2^24 workgroups of the carry
    assert workspace(1, 2 ** 14 - 1, 1, 64, 1, 128, 64) == 0


@pytest.mark.gpu
def test_linear_attention_up_to_the_limit():
    """Just below the limits: 2^24 - 64 and 2^23 - 64 workgroups."""
    if not torch.cuda.is_available():
        pytest.skip("no ROCm GPU visible")
    one = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    b, H, g = 2 ** 18 - 1, 64, torch.zeros(64, device="cuda")
    state = one(b, H, 1, 1)
    o = api.ssm_linattn_step(state, one(b, 1, 1), one(b, 1, 1), one(b, H, 1), g)
    assert bool((o == 2).all()) and bool((state == 2).all())
    b = 2 ** 17 - 1
    o, _ = api.ssm_linattn_fwd(one(b, 1, 1, 4), one(b, 1, 1, 4), one(b, 1, H, 4), g, return_final_state=False)
    assert bool((o == 4).all())
    with pytest.raises(api.SsmError) as e:
        api.ssm_linattn_fwd(one(b + 1, 1, 1, 4), one(b + 1, 1, 1, 4), one(b + 1, 1, H, 4), g, return_final_state=False)
    assert e.value.status == SHAPE


@pytest.mark.gpu
def test_no_steps_and_a_state_of_more_than_2_to_the_32_elements():
    if not torch.cuda.is_available():
        pytest.skip("no ROCm GPU visible")
    b, H, N, P = 520, 64, 128, 1024  # 4.4e9 elements
    z = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    S = torch.full((b, H, P, N), 7.0, device="cuda")
    api.ssm_linattn_fwd(z(b, 0, 1, N), z(b, 0, 1, N), z(b, 0, H, P), z(H), final_state=S)
    assert all(not bool(S[i].any()) for i in (0, 1, 255, 256, 257, 511, 512, 518, 519))


def test_norm_launches():
    for d, most in ((1, 2 ** 24), (4096, 2 ** 24), (4097, 2 ** 22), (16384, 2 ** 22)):
        for rows in (most, 2 * most):
            assert norm_fwd(rows=rows, d=d, w_rows=most) == SHAPE
            assert norm_bwd(rows=rows, d=d, w_rows=most) == SHAPE
            assert api.lib().ssm_layernorm_bwd_workspace(rows, d, most, ctypes.byref(I64())) == SHAPE
        assert api.lib().ssm_layernorm_bwd_workspace(most - 1, d, most - 1, ctypes.byref(I64())) == 0


@pytest.mark.gpu
def test_norm_of_many_weight_rows():
    """2^22 and more pieces of 16 columns in the sum of the partial rows; weight rows that have one row each, so dw and dbias
    are dy·x̂ and dy; and the zeros of a call without rows, 2^32 of them."""
    if not torch.cuda.is_available():
        pytest.skip("no ROCm GPU visible")
    for rows, d in ((32768, 2048), (32770, 2050)):
        x = torch.randn(rows, d, generator=torch.Generator(device="cuda").manual_seed(d), device="cuda").bfloat16()
        w = torch.ones(rows, d, device="cuda")
        _, m, r = api.ssm_layernorm_fwd(x, w, return_stats=True)
        g = api.ssm_layernorm_bwd(x, w, dy=x, mean=m, rstd=r)
        assert torch.equal(g["dbias"], x.float())
        want = x.double() * ((x.double() - m.double()[:, None]) * r.double()[:, None])
        # x̂ takes two roundings after that of the difference, the product one
        tol = 2.0 ** -24 * (2 * x.double().abs() * (x.double().abs() + m.double().abs()[:, None]) * r.double()[:, None] +
                            3 * want.abs())
        assert bool(((g["dw"].double() - want).abs() <= tol).all())
        del x, w, g, want, tol
    rows = 2 ** 24 - 1
    x = torch.ones(rows, 2, device="cuda")
    assert torch.equal(api.ssm_layernorm_fwd(x, x), torch.zeros_like(x))
    with pytest.raises(api.SsmError) as e:
        big = torch.ones(rows + 1, 2, device="cuda")
        api.ssm_layernorm_fwd(big, big)
    assert e.value.status == SHAPE
    k, d = 2 ** 20, 4096
    w, none = torch.ones(k, d, device="cuda"), torch.empty(0, k, d, device="cuda")
    dw = torch.full((k, d), 5.0, device="cuda")
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    assert api.lib().ssm_layernorm_bwd(p(none), p(w), p(none), None, None, None, p(dw), None, 0, d, k, 0, 0, 0, None, 0,
                                       api._stream(w.device)) == 0
    assert not bool(dw[:: 2 ** 18].any()) and not bool(dw[-1].any()) and not bool(dw[k // 2:].any())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,d,k", [(700, 64, 1), (3000, 130, 2), (2100, 2048, 1), (1200, 5000, 4)])
def test_norm_gradient_in_place(rows, d, k, dtype):
    """dx written over x, or over dy, as the header allows, with more rows than workgroups."""
    if not torch.cuda.is_available():
        pytest.skip("no ROCm GPU visible")
    r = torch.Generator(device="cuda").manual_seed(d)
    n = lambda *s: torch.randn(s, generator=r, device="cuda")  # noqa: E731
    x, dy, w = n(rows // k, k, d).to(dtype), n(rows // k, k, d).to(dtype), n(k, d)
    _, m, rs = api.ssm_layernorm_fwd(x, w, return_stats=True)
    want = api.ssm_layernorm_bwd(x, w, dy=dy, mean=m, rstd=rs)
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    for over in ("x", "dy"):
        a, c, dw, db = x.clone(), dy.clone(), torch.empty_like(w), torch.empty_like(w)
        dx = a if over == "x" else c
        assert api.lib().ssm_layernorm_bwd(p(a), p(w), p(c), p(m), p(rs), p(dx), p(dw), p(db), rows, d, k, 0, 0,
                                           0 if dtype == torch.float32 else 1, None, 0, api._stream(x.device)) == 0
        torch.cuda.synchronize()
        assert torch.equal(dx, want["dx"]) and torch.equal(dw, want["dw"]) and torch.equal(db, want["dbias"]), over

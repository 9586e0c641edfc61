"""Refusals of softmax attention, its paged cache and the position rotation at the C ABI and in the binding: bad arguments
are rejected on the host before any launch (no GPU needed; the fake pointers below are never dereferenced)."""
import ctypes
import math

import pytest
import torch

from selective_state_space_82_amd import api

NULL, SHAPE, UNSUPPORTED, ALIAS, SCRATCH = 1, 2, 3, 5, 6
I64 = ctypes.c_int64


def at(i, off=0):
    return ctypes.c_void_p(0x10000000 * (i + 1) + off)


def rows(b=1, Lq=64, Lk=None, cu=False, **kw):
    r = api.AttnRows()
    r.b, r.Lq, r.Lk = b, Lq, Lq if Lk is None else Lk
    if cu:
        r.cu_q, r.cu_k, r.tokens_q, r.tokens_k = at(60), at(61), b * r.Lq, b * r.Lk
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def fwd(r=None, H=2, G=1, D=16, dtype=0, scale=0.25, strides=None, ws=None, ws_bytes=0, **ptr):
    p = {n: at(i) for i, n in enumerate(("q", "k", "v", "o", "lse"))}
    p.update(ptr)
    r = rows() if r is None else r
    return api.lib().ssm_attn_fwd(p["q"], p["k"], p["v"], scale, 1, ctypes.byref(r), p["o"], p["lse"], H, G, D, dtype, strides, ws,
                                  ws_bytes, None)


def bwd(r=None, H=2, G=1, D=16, dtype=0, scale=0.25, strides=None, ws=None, ws_bytes=0, **ptr):
    p = {n: at(i) for i, n in enumerate(("q", "k", "v", "o", "lse", "do", "dq", "dk", "dv"))}
    p.update(ptr)
    r = rows() if r is None else r
    return api.lib().ssm_attn_bwd(p["q"], p["k"], p["v"], p["o"], p["lse"], p["do"], scale, 1, ctypes.byref(r), p["dq"], p["dk"],
                                  p["dv"], H, G, D, dtype, strides, ws, ws_bytes, None)


def pages(n=8, size=16, most=4, k_page=0, v_page=0, table=at(50)):
    return api.Pages(table, n, size, most, k_page, v_page)


def step(g=None, b=2, H=2, G=1, D=16, dtype=0, scale=0.25, max_len=0, ws=None, ws_bytes=0, q_b=0, q_h=0, **ptr):
    p = {n: at(i) for i, n in enumerate(("q", "k", "v", "len", "o", "lse"))}
    p.update(ptr)
    g = pages() if g is None else g
    return api.lib().ssm_attn_step(p["q"], p["k"], p["v"], ctypes.byref(g), p["len"], scale, p["o"], p["lse"], b, H, G, D, q_b, q_h,
                                   max_len, dtype, ws, ws_bytes, None)


def append(g=None, t=None, H=2, G=1, D=16, dtype=0, rotary=16, strides=None, **ptr):
    p = {n: at(i) for i, n in enumerate(("q", "k", "v", "q_out", "k_out", "k_cache", "v_cache", "len", "freq"))}
    p.update(ptr)
    g = pages() if g is None else g
    t = api.Tokens(None, None, 2, 1, 2) if t is None else t
    return api.lib().ssm_kv_append(p["q"], p["k"], p["v"], p["q_out"], p["k_out"], p["k_cache"], p["v_cache"], ctypes.byref(g),
                                   p["len"], ctypes.byref(t), p["freq"], rotary, 0, H, G, D, dtype, strides, None)


def rope(t=None, H=2, D=16, dtype=0, rotary=16, s=(0, 0, 0), **ptr):
    p = {"x": at(0), "out": at(1), "len": None, "freq": at(2)}
    p.update(ptr)
    t = api.Tokens(None, None, 2, 1, 2) if t is None else t
    return api.lib().ssm_rope(p["x"], p["out"], p["len"], ctypes.byref(t), p["freq"], rotary, 0, 0, H, D, *s, dtype, None)


@pytest.mark.parametrize("call,names", [(fwd, ("q", "k", "v", "o")),
                                        (bwd, ("q", "k", "v", "o", "lse", "do", "dq", "dk", "dv")),
                                        (step, ("q", "k", "v", "len", "o")),
                                        (append, ("k", "v", "k_cache", "v_cache", "len")), (rope, ("x", "out", "freq"))])
def test_null_pointers(call, names):
    for n in names:
        assert call(**{n: None}) == NULL, n


def test_null_descriptors():
    lib, n = api.lib(), I64()
    assert append(q=None) == NULL and append(q_out=None) == NULL  # both or neither
    assert step(pages(table=None)) == NULL and append(pages(table=None)) == NULL
    assert fwd(rows(cu=True, cu_k=None)) == NULL and bwd(rows(cu=True, cu_q=None)) == NULL
    assert lib.ssm_attn_fwd_workspace(None, 1, 1, 8, 0, ctypes.byref(n)) == NULL
    assert lib.ssm_attn_fwd_workspace(ctypes.byref(rows()), 1, 1, 8, 0, None) == NULL
    assert lib.ssm_attn_bwd_workspace(ctypes.byref(rows()), 1, 1, 8, None) == NULL
    assert lib.ssm_attn_step_workspace(1, 1, 1, 8, None, 0, ctypes.byref(n)) == NULL
    assert lib.ssm_attn_step_workspace(1, 1, 1, 8, ctypes.byref(pages()), 0, None) == NULL


@pytest.mark.parametrize("call", [fwd, bwd, step, append, rope])
@pytest.mark.parametrize("kw,code", [({"H": 0}, SHAPE), ({"D": 0}, SHAPE), ({"D": 129}, UNSUPPORTED),
                                     ({"dtype": 2}, UNSUPPORTED), ({"H": 1 << 24}, SHAPE)])
def test_heads(call, kw, code):
    assert call(**kw) == code
    if call is not rope:
        assert call(G=0) == SHAPE and call(H=3, G=2) == SHAPE


@pytest.mark.parametrize("call", [fwd, bwd, step])
def test_scale(call):
    for s in (math.nan, math.inf, -math.inf):
        assert call(scale=s) == UNSUPPORTED


@pytest.mark.parametrize("call", [fwd, bwd])
def test_rows(call):
    for r in (rows(b=0), rows(Lq=-1), rows(Lk=-1), rows(Lq=(1 << 30) + 1), rows(Lk=(1 << 30) + 1), rows(b=1 << 40),
              rows(b=1 << 16, Lq=1 << 30), rows(cu=True, tokens_q=-1), rows(cu=True, tokens_k=1 << 31),
              rows(b=1 << 24, Lq=128)):
        assert call(r) == SHAPE, {n: getattr(r, n) for n, _ in r._fields_}


def test_strides():
    for name, v in (("q_t", -1), ("k_h", -1), ("v_t", (1 << 24) + 1), ("q_b", 1 << 41)):
        s = api.LinAttnStrides()
        setattr(s, name, v)
        assert fwd(rows(b=2), strides=ctypes.byref(s)) == SHAPE, name
        assert bwd(rows(b=2), strides=ctypes.byref(s)) == SHAPE, name
    assert step(q_b=-1) == SHAPE and rope(s=(-1, 0, 0)) == SHAPE
    # a strided input reaches as far as its strides say
    s = api.LinAttnStrides()
    s.q_b = 0x1000000 // 4
    assert fwd(rows(b=2), strides=ctypes.byref(s), o=ctypes.c_void_p(0x10000000 + 0x1000000)) == ALIAS


def test_aliasing():
    for out in ("o", "lse"):
        for other in ("q", "k", "v"):
            assert fwd(**{out: at(30), other: at(30)}) == ALIAS, (out, other)
    assert fwd(o=at(30), lse=at(30)) == ALIAS
    assert fwd(rows(len_q=at(30)), o=at(30)) == ALIAS and fwd(rows(cu=True, cu_k=at(30)), lse=at(30)) == ALIAS
    outs = ("dq", "dk", "dv")
    for out in outs:
        for other in ("q", "k", "v", "o", "lse", "do") + outs:
            if other != out:
                assert bwd(**{out: at(30), other: at(30)}) == ALIAS, (out, other)
    for out in ("o", "lse"):
        for other in ("q", "k", "v", "len"):
            assert step(**{out: at(30), other: at(30)}) == ALIAS, (out, other)
    assert step(pages(table=at(30)), o=at(30)) == ALIAS
    for out in ("q_out", "k_out", "k_cache", "v_cache"):
        for other in ("v", "len", "freq") + (("k",) if out != "k_out" else ()) + (("q",) if out != "q_out" else ()):
            assert append(**{out: at(30), other: at(30)}) == ALIAS, (out, other)
        for other in ("q_out", "k_out", "k_cache", "v_cache"):
            if other != out:
                assert append(**{out: at(30), other: at(30)}) == ALIAS, (out, other)
    assert append(q_out=at(0, 16)) == ALIAS  # part of q
    s = api.LinAttnStrides(0, 0, 20, 0, 0, 16, 0, 0, 16)
    assert append(q_out=at(0), strides=ctypes.byref(s)) == ALIAS  # in place needs dense rows
    assert rope(out=at(0, 16)) == ALIAS and rope(out=at(0), s=(40, 0, 16)) == ALIAS and rope(out=at(2)) == ALIAS


def test_pools():
    """Both caches in one pool, page about, and pools whose pages would overlap."""
    page = 16 * 16 * 4  # bytes
    one = dict(k_cache=at(20), v_cache=at(20, page))
    assert append(pages(k_page=2 * 256, v_page=2 * 256), **one, freq=None, q=None, q_out=None, k_out=None,
                  t=api.Tokens(None, None, 1, 0, 0)) == 0
    assert append(pages(k_page=2 * 256, v_page=2 * 256), k_cache=at(20), v_cache=at(20, page - 4)) == ALIAS
    assert append(pages(k_page=2 * 256, v_page=2 * 256 + 4), **one) == ALIAS
    assert append(pages(k_page=256), **one) == ALIAS


@pytest.mark.parametrize("call", [step, append])
def test_pages(call):
    for kw in ({"n": 0}, {"size": 0}, {"most": 0}, {"n": 1 << 31}, {"size": (1 << 20) + 1}, {"size": 1 << 20, "most": 1 << 11},
               {"k_page": -1}, {"v_page": 255}, {"k_page": 1 << 40}):
        assert call(pages(**kw)) == SHAPE, kw


def test_tokens_and_rotation():
    T = api.Tokens
    for t in (T(None, None, 0, 1, 0), T(None, None, 2, 3, 5), T(None, None, 2, -1, -2), T(at(40), None, 2, 0, -1),
              T(None, None, 1 << 31, 1, 1 << 31)):
        assert append(t=t) == SHAPE and rope(t=t) == SHAPE
    for r in (0, 1, 15, 17, 18, -2):
        assert append(rotary=r) == SHAPE and rope(rotary=r) == SHAPE


def test_workspace():
    lib, n = api.lib(), I64()
    r = rows(b=1, Lq=4096)
    assert lib.ssm_attn_fwd_workspace(ctypes.byref(r), 2, 1, 16, 0, ctypes.byref(n)) == 0 and n.value > 0
    assert fwd(r, ws=at(40), ws_bytes=n.value - 1) == SCRATCH
    assert fwd(r, ws=at(40, 8), ws_bytes=n.value) == UNSUPPORTED
    assert fwd(r, ws=at(40), ws_bytes=n.value, o=at(40)) == ALIAS and fwd(r, ws=at(40), ws_bytes=n.value, k=at(40)) == ALIAS
    assert lib.ssm_attn_bwd_workspace(ctypes.byref(r), 2, 1, 16, ctypes.byref(n)) == 0 and n.value > 0
    assert bwd(r, ws=at(40), ws_bytes=n.value - 1) == SCRATCH
    assert bwd(r, ws=at(40), ws_bytes=n.value, dv=at(40)) == ALIAS
    assert lib.ssm_attn_step_workspace(2, 2, 1, 16, ctypes.byref(pages(most=64)), 0, ctypes.byref(n)) == 0 and n.value > 0
    assert step(pages(most=64), ws=at(40), ws_bytes=n.value - 1) == SCRATCH
    assert step(pages(most=64), ws=at(40), ws_bytes=n.value, q=at(40)) == ALIAS
    # calls that fill the device are not cut
    assert lib.ssm_attn_fwd_workspace(ctypes.byref(rows(b=8, Lq=4096)), 32, 8, 128, 1, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.ssm_attn_step_workspace(512, 32, 8, 128, ctypes.byref(pages(most=64, size=64)), 0, ctypes.byref(n)) == 0
    assert n.value == 0


def test_binding_refuses():
    q, k = torch.zeros(1, 4, 2, 8), torch.zeros(1, 4, 1, 8)
    cache, i32 = torch.zeros(2, 16, 1, 8), torch.zeros(1, dtype=torch.int32)
    for call in (lambda: api.ssm_attn_fwd(q, k, k), lambda: api.ssm_rope(q, torch.ones(4, dtype=torch.float64)),
                 lambda: api.ssm_attn_bwd(q, k, k, o=q, lse=q[..., 0], do=q),
                 lambda: api.ssm_attn_step(q[:, 0], cache, cache, i32[None], i32),
                 lambda: api.ssm_kv_append(k[:, 0], k[:, 0], cache, cache, i32[None], i32)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    if not torch.cuda.is_available():
        return
    q, k, cache, i32 = q.cuda(), k.cuda(), cache.cuda(), i32.cuda()
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    f = torch.ones(4, dtype=torch.float64, device="cuda")
    bad = [lambda: api.ssm_attn_fwd(q[0], k[0], k[0]), lambda: api.ssm_attn_fwd(q, k[0], k[0]),
           lambda: api.ssm_attn_fwd(q, k, k, cu_seqlens=cu, max_len=4), lambda: api.ssm_attn_fwd(q[0], k[0], k[0], cu_seqlens=cu),
           lambda: api.ssm_attn_fwd(q[0], k[0], k[0], cu_seqlens=cu, max_len=4, lengths=i32),
           lambda: api.ssm_attn_fwd(q[0], k[0], k[0], cu_seqlens=cu, max_len=4, max_len_k=4),
           lambda: api.ssm_attn_fwd(q, k[:, :2], k[:, :2], lengths=i32), lambda: api.ssm_attn_fwd(q, k, k[:, :2]),
           lambda: api.ssm_attn_fwd(q, k, k, lengths=cu), lambda: api.ssm_attn_fwd(q, k[..., :4], k[..., :4]),
           lambda: api.ssm_attn_fwd(q.transpose(2, 3), q.transpose(2, 3), q.transpose(2, 3)),
           lambda: api.ssm_attn_step(q, cache, cache, i32[None], i32), lambda: api.ssm_attn_step(q[:, 0], cache, cache, i32, i32),
           lambda: api.ssm_attn_step(q[:, 0], cache.transpose(1, 2), cache, i32[None], i32),
           lambda: api.ssm_attn_step(q[:, 0], cache, cache, i32[None], cu),
           lambda: api.ssm_kv_append(k, k, cache, cache.clone(), i32[None], i32, cu_seqlens=cu),
           lambda: api.ssm_kv_append(k[:, 0], k[:, 0], cache, cache.clone(), i32[None], i32, q_out=q[:, 0]),
           lambda: api.ssm_kv_append(k[:, 0], k[:, 0], cache, cache.clone(), i32[None], i32, new_lengths=i32),
           lambda: api.ssm_rope(q, f[:0]), lambda: api.ssm_rope(q, torch.ones(5, dtype=torch.float64, device="cuda"))]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(i)
    for call in (lambda: api.ssm_attn_fwd(q, k, k.bfloat16()), lambda: api.ssm_attn_fwd(q.half(), k.half(), k.half()),
                 lambda: api.ssm_attn_fwd(q, k, k, lengths=i32.long()), lambda: api.ssm_rope(q, f.float()),
                 lambda: api.ssm_attn_bwd(q, k, k, o=q, lse=None, do=q),
                 lambda: api.ssm_attn_step(q[:, 0], cache, cache, i32[None], None)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(api.SsmError):
        api.ssm_kv_append(k[:, 0], k[:, 0], cache, cache, i32[None], i32)  # one cache for both

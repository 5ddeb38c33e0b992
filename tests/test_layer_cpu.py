"""Refusals of the layer operators' C entry points, decided on the host before
any device call (the pointers are fake), and random arguments that must end
in a documented status."""
import math

import pytest
from hypothesis import given, strategies as st

import nvfp4_block_scaled_amax_amd as mxq
from test_abi_cpu import status_of
from test_abi_fuzz import ERRORS, SETTINGS, ptrs, sizes, status

A, B1, B2, B3, B4, B5, B6, B7, B8 = ((k + 1) << 20 for k in range(9))
BF, F4 = mxq.MXQ_OUT_BF16, mxq.MXQ_OUT_F32
GOOD = dict(top_k=4, n_groups=1, topk_groups=1, group_topk=1, scoring=mxq.MXQ_SCORE_SOFTMAX,
            renormalize=1, scale=1.0)


def route(dtype=F4, logits=A, bias=None, T=8, E=16, w=B1, e=B2, tr=B3, rt=B4, seg=B5, ws=B6,
          nbytes=1 << 20, **p):
    return status_of(mxq.mxq_moe_route, dtype, logits, bias, T, E, dict(GOOD, **p), w, e, tr, rt,
                     seg, ws, nbytes, 0)


def test_route_refusals():
    assert route(dtype=2) == mxq.MXQ_ERR_ARG
    assert route(logits=None) == mxq.MXQ_ERR_NULL
    assert route(e=None) == mxq.MXQ_ERR_NULL
    assert route(tr=None) == mxq.MXQ_ERR_OFFSETS
    assert route(seg=None) == mxq.MXQ_ERR_OFFSETS
    assert route(scoring=2) == mxq.MXQ_ERR_ARG
    assert route(group_topk=0) == mxq.MXQ_ERR_ARG
    assert route(group_topk=3) == mxq.MXQ_ERR_ARG
    assert route(scale=math.inf) == mxq.MXQ_ERR_ARG
    assert route(scale=math.nan) == mxq.MXQ_ERR_ARG
    assert route(top_k=0) == mxq.MXQ_ERR_SIZE
    assert route(top_k=17) == mxq.MXQ_ERR_SIZE
    assert route(E=128, top_k=65) == mxq.MXQ_ERR_SIZE
    assert route(E=1025) == mxq.MXQ_ERR_SIZE
    assert route(T=0) == mxq.MXQ_ERR_SIZE
    assert route(T=1 << 24) == mxq.MXQ_ERR_SIZE
    assert route(T=(1 << 24) - 1, E=128, top_k=64, nbytes=1 << 40) == mxq.MXQ_ERR_DEVICE
    assert route(n_groups=3) == mxq.MXQ_ERR_SHAPE
    assert route(n_groups=4, topk_groups=5) == mxq.MXQ_ERR_SIZE
    assert route(E=130, n_groups=65) == mxq.MXQ_ERR_SIZE
    assert route(ws=None) == mxq.MXQ_ERR_NULL
    assert route(nbytes=0) == mxq.MXQ_ERR_SIZE
    assert route(ws=B6 + 8) == mxq.MXQ_ERR_ALIGN
    assert route(logits=A + 2) == mxq.MXQ_ERR_ALIGN
    assert route(dtype=BF, logits=A + 1) == mxq.MXQ_ERR_ALIGN
    assert route() == mxq.MXQ_ERR_DEVICE
    assert route(tr=None, rt=None, seg=None, ws=None, nbytes=0) == mxq.MXQ_ERR_DEVICE
    assert mxq.mxq_moe_route_workspace(8, 16) > 0
    for T, E in ((0, 16), (8, 0), (8, 1025), (1 << 24, 16), (-1, 4)):
        assert mxq.mxq_moe_route_workspace(T, E) == 0


def test_route_backward_refusals():
    def bwd(dtype=F4, dw=A, x=B1, e=B2, T=8, E=16, k=4, scoring=0, scale=1.0, d=B3):
        return status_of(mxq.mxq_moe_route_backward, dtype, dw, x, e, T, E, k, scoring, True,
                         scale, d, 0)
    assert bwd(dtype=7) == mxq.MXQ_ERR_ARG
    assert bwd(scoring=-1) == mxq.MXQ_ERR_ARG
    assert bwd(scale=-math.inf) == mxq.MXQ_ERR_ARG
    assert bwd(e=None) == mxq.MXQ_ERR_NULL
    assert bwd(k=0) == mxq.MXQ_ERR_SIZE
    assert bwd(k=65) == mxq.MXQ_ERR_SIZE
    assert bwd(E=1025) == mxq.MXQ_ERR_SIZE
    assert bwd(e=B2 + 4) == mxq.MXQ_ERR_ALIGN
    assert bwd() == mxq.MXQ_ERR_DEVICE


def test_combine_refusals():
    def fwd(dtype=BF, rows=A, R=64, tr=B1, w=B2, T=8, k=4, cols=32, od=BF, out=B3):
        return status_of(mxq.mxq_moe_combine, dtype, rows, R, tr, w, T, k, cols, od, out, 0)

    def bwd(dtype=BF, d=A, rows=B1, R=64, tr=B2, w=B3, seg=None, G=0, T=8, k=4, cols=32, dr=B4,
            dw=B5):
        return status_of(mxq.mxq_moe_combine_backward, dtype, d, rows, R, tr, w, seg, G, T, k,
                         cols, dr, dw, 0)
    for f in (fwd, bwd):
        assert f(dtype=3) == mxq.MXQ_ERR_ARG
        assert f(rows=None) == mxq.MXQ_ERR_NULL
        assert f(tr=None) == mxq.MXQ_ERR_NULL
        assert f(R=0) == mxq.MXQ_ERR_SIZE
        assert f(T=0) == mxq.MXQ_ERR_SIZE
        assert f(T=1 << 24) == mxq.MXQ_ERR_SIZE
        assert f(k=0) == mxq.MXQ_ERR_SIZE
        assert f(k=65) == mxq.MXQ_ERR_SIZE
        assert f(cols=0) == mxq.MXQ_ERR_SIZE
        assert f(cols=12) == mxq.MXQ_ERR_SHAPE
        assert f(cols=1 << 61, R=8) == mxq.MXQ_ERR_SIZE
        assert f(rows=(1 << 21) + 8) == mxq.MXQ_ERR_ALIGN
        assert f() == mxq.MXQ_ERR_DEVICE
    assert fwd(od=2) == mxq.MXQ_ERR_ARG
    assert bwd(seg=B6, G=0) == mxq.MXQ_ERR_SIZE
    assert bwd(seg=B6 + 4, G=3) == mxq.MXQ_ERR_ALIGN


def test_matvec_refusals():
    def mv(fmt=0, x=A, xb=None, xs=None, b=B1, bb=B2, bs=B3, rpb=1, M=4, N=8, K=64, od=BF, c=B4):
        return status_of(mxq.mxq_nvfp4_matvec, fmt, x, xb, xs, b, bb, bs, rpb, M, N, K, od, c, 0)

    def ex(fmt=0, x=A, xb=None, xs=None, b=B1, bb=B2, bs=B3, seg=B4, G=2, M=4, N=8, K=64, od=BF,
           c=B5):
        return status_of(mxq.mxq_nvfp4_expert_matvec, fmt, x, xb, xs, b, bb, bs, seg, G, M, N, K,
                         od, c, 0)

    def gu(fmt=0, x=A, xb=None, xs=None, T=4, rt=B1, seg=B2, G=2, M=4, b=B3, bb=B4, u=B5, ub=B6,
           s=B7, N=8, K=64, od=BF, c=B8):
        return status_of(mxq.mxq_nvfp4_expert_gateup, fmt, x, xb, xs, T, rt, seg, G, M, b, bb, u,
                         ub, s, N, K, od, c, 0)
    for f in (mv, ex, gu):
        assert f(fmt=3) == mxq.MXQ_ERR_ARG
        assert f(od=2) == mxq.MXQ_ERR_ARG
        assert f(x=None) == mxq.MXQ_ERR_NULL
        assert f(fmt=2) == mxq.MXQ_ERR_NULL
        assert f(fmt=2, xb=A + 8) == mxq.MXQ_ERR_NULL
        assert f(xb=A) == mxq.MXQ_ERR_OFFSETS
        assert f(fmt=1, xs=A) == mxq.MXQ_ERR_OFFSETS
        assert f(b=None) == mxq.MXQ_ERR_NULL
        assert f(c=None) == mxq.MXQ_ERR_NULL
        assert f(M=0) == mxq.MXQ_ERR_SIZE
        assert f(N=0) == mxq.MXQ_ERR_SIZE
        assert f(N=(1 << 24) + 1) == mxq.MXQ_ERR_SIZE
        assert f(K=0) == mxq.MXQ_ERR_SIZE
        assert f(K=96) == mxq.MXQ_ERR_SHAPE
        assert f(K=(1 << 16) + 64) == mxq.MXQ_ERR_SIZE
        assert f(x=A + 8) == mxq.MXQ_ERR_ALIGN
        assert f(b=A + 8) == mxq.MXQ_ERR_ALIGN
        assert f(bb=A + 2) == mxq.MXQ_ERR_ALIGN
        assert f(c=A + 1) == mxq.MXQ_ERR_ALIGN
        assert f() == mxq.MXQ_ERR_DEVICE
    assert mv(M=65) == mxq.MXQ_ERR_SIZE
    assert mv(rpb=0) == mxq.MXQ_ERR_SIZE
    for f in (ex, gu):
        assert f(seg=None) == mxq.MXQ_ERR_NULL
        assert f(G=0) == mxq.MXQ_ERR_SIZE
        assert f(G=(1 << 16) + 1) == mxq.MXQ_ERR_SIZE
        assert f(G=1 << 16, N=1 << 24) == mxq.MXQ_ERR_SIZE
        assert f(M=(1 << 30) + 1) == mxq.MXQ_ERR_SIZE
        assert f(seg=A + 4) == mxq.MXQ_ERR_ALIGN
    assert gu(rt=None) == mxq.MXQ_ERR_NULL
    assert gu(u=None) == mxq.MXQ_ERR_NULL
    assert gu(T=0) == mxq.MXQ_ERR_SIZE


def test_attention_refusals():
    def at(q=A, k=(B1, B2, B3), v=(B4, B5, B6), table=B7, lens=B8, S=2, Q=1, H=8, Hkv=2, D=128,
           n_pages=4, page=16, max_pages=2, scale=0.1, causal=True, window=0, out=B8 + (1 << 20),
           lse=None, ws=B8 + (1 << 21), nbytes=1 << 60):
        return status_of(mxq.mxq_nvfp4_attention, q, k, v, table, lens, S, Q, H, Hkv, D, n_pages,
                         page, max_pages, scale, causal, window, out, lse, ws, nbytes, 0)
    assert at(q=None) == mxq.MXQ_ERR_NULL
    assert at(k=None) == mxq.MXQ_ERR_NULL
    assert at(v=(B4, None, B6)) == mxq.MXQ_ERR_NULL
    assert at(lens=None) == mxq.MXQ_ERR_NULL
    for scale in (0.0, -1.0, math.inf, math.nan):
        assert at(scale=scale) == mxq.MXQ_ERR_ARG
    assert at(window=-1) == mxq.MXQ_ERR_ARG
    assert at(causal=False, window=3) == mxq.MXQ_ERR_ARG
    for bad in (dict(S=0), dict(Q=0), dict(H=0), dict(Hkv=0), dict(n_pages=0), dict(page=0),
                dict(max_pages=0), dict(S=1 << 25), dict(Q=1 << 40, S=1 << 40),
                dict(n_pages=1 << 50), dict(max_pages=1 << 28), dict(page=1 << 40)):
        assert at(**bad) == mxq.MXQ_ERR_SIZE, bad
    assert at(D=96) == mxq.MXQ_ERR_SHAPE
    assert at(Hkv=3) == mxq.MXQ_ERR_SHAPE
    assert at(page=24) == mxq.MXQ_ERR_SHAPE
    assert at(q=A + 8) == mxq.MXQ_ERR_ALIGN
    assert at(k=(B1 + 8, B2, B3)) == mxq.MXQ_ERR_ALIGN
    assert at(k=(B1, B2 + 4, B3)) == mxq.MXQ_ERR_ALIGN
    assert at(v=(B4, B5, B6 + 4)) == mxq.MXQ_ERR_ALIGN
    assert at(table=B7 + 4) == mxq.MXQ_ERR_ALIGN
    assert at() == mxq.MXQ_ERR_DEVICE
    ws = mxq.mxq_nvfp4_attention_workspace
    assert ws(0, 1, 8, 2, 128, 64) == 0 and ws(2, 1, 8, 3, 128, 64) == 0
    assert ws(2, 1, 8, 2, 96, 64) == 0 and ws(2, 1, 8, 2, 128, 1 << 40) == 0


@SETTINGS
@given(p=st.lists(ptrs, min_size=14, max_size=14), a=sizes, b=sizes, c=sizes, d=sizes, e=sizes,
       f=sizes, dt=st.integers(-1, 2), g=st.integers(-1, 3))
def test_random_arguments(p, a, b, c, d, e, f, dt, g):
    par = dict(top_k=c, n_groups=d, topk_groups=e, group_topk=g, scoring=dt, renormalize=0,
               scale=1.0)
    calls = [
        (mxq.mxq_moe_route, dt, p[0], p[1], a, b, par, p[2], p[3], p[4], p[5], p[6], p[7], f, 0),
        (mxq.mxq_moe_route_backward, dt, p[0], p[1], p[2], a, b, c, g, True, 1.0, p[3], 0),
        (mxq.mxq_moe_combine, dt, p[0], a, p[1], p[2], b, c, d, g, p[3], 0),
        (mxq.mxq_moe_combine_backward, dt, p[0], p[1], a, p[2], p[3], p[4], e, b, c, d, p[5],
         p[6], 0),
        (mxq.mxq_nvfp4_matvec, g, p[0], p[1], p[2], p[3], p[4], p[5], a, b, c, d, dt, p[6], 0),
        (mxq.mxq_nvfp4_expert_matvec, g, p[0], p[1], p[2], p[3], p[4], p[5], p[6], a, b, c, d, dt,
         p[7], 0),
        (mxq.mxq_nvfp4_expert_gateup, g, p[0], p[1], p[2], e, p[3], p[4], a, b, p[5], p[6], p[7],
         p[8], p[9], c, d, dt, p[10], 0),
        (mxq.mxq_nvfp4_attention, p[0], tuple(p[1:4]), tuple(p[4:7]), p[7], p[8], a, b, c, d,
         128, e, 16, f, 0.5, True, max(dt, 0), p[9], p[10], p[11], a, 0),
    ]
    for fn, *args in calls:
        assert status(fn, *args) in ERRORS, fn.__name__
    assert mxq.mxq_moe_route_workspace(a, b) >= 0
    assert mxq.mxq_nvfp4_attention_workspace(a, b, c, d, 128, e) >= 0

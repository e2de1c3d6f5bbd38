"""Refusals of the routing, row and adapter entry points: all before anything is enqueued, no GPU needed."""
import pytest
import torch

import dense_gemm_09_amd as g
from dense_gemm_09_amd import OUT_BF16, OUT_F32

OK, NULLP, BAD_DIM, BAD_LD, BAD_ENUM, UNSUP, SMALL = range(7)
FAKE = 0x7F0000000000


def route(T=8, E=64, k=4, x=FAKE, ld=None, t=OUT_F32, score=0, bias=None, groups=1, top=1, best=1, ids=FAKE, w=FAKE):
    return g.lib().gemm_route(T, E, k, x, E if ld is None else ld, t, score, bias, groups, top, best, 0, 1.0, ids, w, None)


def test_route_refusals():
    assert route(t=2) == BAD_ENUM and route(score=2) == BAD_ENUM
    for bad in (dict(T=-1), dict(T=(1 << 30) + 1), dict(E=0), dict(k=0), dict(k=65), dict(groups=0), dict(groups=3),
                dict(groups=4, top=5), dict(groups=4, top=0), dict(best=0), dict(best=3), dict(groups=32, top=1, k=3)):
        assert route(**bad) == BAD_DIM, bad
    assert route(E=1025) == UNSUP and route(k=33) == UNSUP and route(E=1024, groups=128, top=128) == UNSUP
    assert route(ld=63) == BAD_LD
    for name in ("x", "ids", "w"):
        assert route(**{name: None}) == NULLP
    assert route(x=FAKE + 2) == UNSUP and route(x=FAKE + 1, t=OUT_BF16) == UNSUP and route(bias=FAKE + 1) == UNSUP
    assert route(T=0, x=None, ids=None, w=None) == OK


def grad(T=8, E=64, k=4, x=FAKE, ld=64, t=OUT_F32, score=0, ids=FAKE, dw=FAKE, dx=FAKE, ldd=64):
    return g.lib().gemm_route_grad(T, E, k, x, ld, t, score, 0, 1.0, ids, dw, dx, ldd, None)


def test_route_grad_refusals():
    assert grad(t=3) == BAD_ENUM and grad(score=-1) == BAD_ENUM
    assert grad(T=-1) == BAD_DIM and grad(k=65) == BAD_DIM and grad(E=0) == BAD_DIM
    assert grad(E=1025, ld=1025, ldd=1025) == UNSUP and grad(k=33) == UNSUP
    assert grad(ld=63) == BAD_LD and grad(ldd=63) == BAD_LD
    for name in ("x", "ids", "dw", "dx"):
        assert grad(**{name: None}) == NULLP
    assert grad(dx=FAKE + 2) == UNSUP
    assert grad(T=0, x=None, ids=None, dw=None, dx=None) == OK


def order(S=100, G=8, e=FAKE, off=FAKE, pos=FAKE, order=None, ws=FAKE, wsb=1 << 30):
    return g.lib().gemm_route_order(S, G, e, off, pos, order, ws, wsb, None)


def test_order_refusals():
    assert order(S=-1) == BAD_DIM and order(S=(1 << 30) + 1) == BAD_DIM and order(G=-1) == BAD_DIM
    assert order(G=8193) == UNSUP and order(e=FAKE + 1) == UNSUP and order(ws=FAKE + 2) == UNSUP
    for name in ("e", "off", "pos"):
        assert order(**{name: None}) == NULLP
    need = g.route_order_workspace_size(100000, 8)
    if need:
        assert order(S=100000, ws=None) == NULLP and order(S=100000, wsb=need - 1) == SMALL
    assert g.route_order_workspace_size(-1, 8) == 0 and g.route_order_workspace_size(8, 8193) == 0


def dispatch(T=4, k=2, R=8, N=16, x=FAKE, ldx=16, size=2, pos=FAKE, y=FAKE, ldy=16):
    return g.lib().gemm_dispatch_rows(T, k, R, N, x, ldx, size, pos, y, ldy, None)


def test_dispatch_refusals():
    assert dispatch(size=3) == BAD_ENUM and dispatch(size=8) == BAD_ENUM
    for bad in (dict(T=-1), dict(R=-1), dict(N=-1), dict(k=0), dict(T=1 << 29, k=3)):
        assert dispatch(**bad) == BAD_DIM, bad
    assert dispatch(k=65) == UNSUP and dispatch(x=FAKE + 1) == UNSUP and dispatch(y=FAKE + 2, size=4) == UNSUP
    assert dispatch(ldx=15) == BAD_LD and dispatch(ldy=15) == BAD_LD
    for name in ("x", "pos", "y"):
        assert dispatch(**{name: None}) == NULLP
    assert dispatch(T=0, x=None) == OK and dispatch(R=0, y=None) == OK and dispatch(N=0, x=None) == OK


def combine(T=4, k=2, R=8, N=16, y=FAKE, ldy=16, yt=1, pos=FAKE, w=None, beta=0.0, c=FAKE, ldc=16, ct=1):
    return g.lib().gemm_combine_rows(T, k, R, N, y, ldy, yt, pos, w, beta, c, ldc, ct, None)


def test_combine_refusals():
    assert combine(yt=2) == BAD_ENUM and combine(ct=-1) == BAD_ENUM
    for bad in (dict(T=-1), dict(R=-1), dict(N=-1), dict(k=0)):
        assert combine(**bad) == BAD_DIM, bad
    assert combine(k=65) == UNSUP and combine(y=FAKE + 1) == UNSUP and combine(c=FAKE + 2, ct=0) == UNSUP
    assert combine(ldy=15) == BAD_LD and combine(ldc=15) == BAD_LD
    for name in ("y", "pos", "c"):
        assert combine(**{name: None}) == NULLP
    assert combine(T=0, c=None) == OK and combine(N=0, c=None) == OK


def combine_grad(T=4, k=2, R=8, N=16, d=FAKE, ldd=16, dt=1, y=FAKE, ldy=16, yt=1, pos=FAKE, dy=FAKE, lddy=16, dw=FAKE):
    return g.lib().gemm_combine_rows_grad(T, k, R, N, d, ldd, dt, y, ldy, yt, pos, None, dy, lddy, dw, None)


def test_combine_grad_refusals():
    assert combine_grad(yt=2) == BAD_ENUM and combine_grad(dt=9) == BAD_ENUM
    assert combine_grad(T=-1) == BAD_DIM and combine_grad(k=65) == UNSUP and combine_grad(dy=FAKE + 1) == UNSUP
    assert combine_grad(ldd=15) == BAD_LD and combine_grad(ldy=15) == BAD_LD and combine_grad(lddy=15) == BAD_LD
    for name in ("d", "y", "pos", "dy"):
        assert combine_grad(**{name: None}) == NULLP
    assert combine_grad(T=0, d=None) == OK and combine_grad(N=0, d=None, dw=None) == OK


def lora(M=8, N=64, K=64, G=2, R=16, a=FAKE, lda=64, b=FAKE, ldb=64, ids=FAKE, down=FAKE, ldd=64, sd=1024, up=FAKE,
         ldu=16, su=1024, scale=None, c=FAKE, ldc=64, ct=1, act=0, ws=FAKE, wsb=1 << 30):
    return g.lib().gemm_lora_bf16(M, N, K, G, R, 1.0, a, lda, b, ldb, ids, down, ldd, sd, up, ldu, su, scale, 0.0, c, ldc,
                                  ct, None, act, ws, wsb, None)


def test_lora_refusals():
    assert lora(ct=2) == BAD_ENUM and lora(act=4) == BAD_ENUM
    for name in ("M", "N", "K", "G", "R"):
        assert lora(**{name: -1}) == BAD_DIM
    assert lora(R=129, ldu=129) == UNSUP and lora(G=65537) == UNSUP
    assert lora(lda=63) == BAD_LD and lora(ldb=63) == BAD_LD and lora(ldc=63) == BAD_LD
    assert lora(ldd=63) == BAD_LD and lora(ldu=15) == BAD_LD and lora(sd=-1) == BAD_LD and lora(su=-1) == BAD_LD
    for name in ("a", "b", "ids", "down", "up", "c", "ws"):
        assert lora(**{name: None}) == NULLP, name
    assert lora(wsb=g.lora_workspace_size(8, 64, 64, 16) - 1) == SMALL
    for bad in (dict(ws=FAKE + 8), dict(a=FAKE + 1), dict(b=FAKE + 1), dict(down=FAKE + 1), dict(up=FAKE + 1),
                dict(ids=FAKE + 2), dict(scale=FAKE + 1), dict(c=FAKE + 1)):
        assert lora(**bad) == UNSUP, bad
    assert lora(M=1 << 20, K=1024, lda=1024, ldb=1024, ldd=1024, wsb=1 << 40) == UNSUP  # A spans 2^31 bytes
    assert lora(M=0, a=None, c=None) == OK and lora(N=0, b=None, c=None) == OK


def test_python_checks():
    """Host tensors and other types are refused before the library is reached."""
    f, i, h = torch.zeros(64), torch.zeros(64, dtype=torch.int32), torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="logits must be a device tensor"):
        g.route(1, 8, 2, f, 8, OUT_F32, g.SCORE_SOFTMAX, None, 1, 1, 1, False, 1.0, i, f)
    with pytest.raises(ValueError, match="expert must be INT32"):
        g.route(1, 8, 2, FAKE, 8, OUT_F32, g.SCORE_SOFTMAX, None, 1, 1, 1, False, 1.0, i.long(), f)
    with pytest.raises(ValueError, match="weight must be FP32"):
        g.route(1, 8, 2, FAKE, 8, OUT_F32, g.SCORE_SOFTMAX, None, 1, 1, 1, False, 1.0, FAKE, h)
    with pytest.raises(ValueError, match="dweight must be FP32"):
        g.route_grad(1, 8, 2, FAKE, 8, OUT_F32, g.SCORE_SOFTMAX, False, 1.0, FAKE, h, FAKE, 8)
    with pytest.raises(ValueError, match="offsets must be INT32"):
        g.route_order(4, 2, FAKE, i.long(), FAKE)
    with pytest.raises(ValueError, match="X must be a device tensor"):
        g.dispatch_rows(2, 2, 4, 8, h, 8, 2, i, h, 8)
    with pytest.raises(ValueError, match="position must be INT32"):
        g.combine_rows(2, 2, 4, 8, FAKE, 8, OUT_BF16, i.long(), None, 0.0, FAKE, 8, OUT_BF16)
    with pytest.raises(ValueError, match="dY must be a device tensor"):
        g.combine_rows_grad(2, 2, 4, 8, FAKE, 8, OUT_BF16, FAKE, 8, OUT_BF16, i, None, h, 8, f)
    with pytest.raises(ValueError, match="adapter must be INT32"):
        g.gemm_lora_bf16(2, 8, 8, 2, 4, 1.0, FAKE, 8, FAKE, 8, i.long(), FAKE, 8, 32, FAKE, 4, 32, None, 0.0, FAKE, 8, OUT_F32)

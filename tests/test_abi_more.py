"""Refusals of the entry points for log probabilities from features, 8-bit integer products and dropout: on the
host, before any device work (no GPU)."""
import ctypes
import os

import pytest

P, Q, O = (ctypes.c_void_p(x) for x in (4096, 4098, 65536))
ODD = ctypes.c_void_p(4097)
BIG = 1 << 60


@pytest.fixture(scope="module")
def L():
    import precision_label_chunk_amd as elmo
    if not os.path.exists(elmo.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return elmo.lib()


def test_linear_logprobs(L):
    def call(**kw):
        a = {**dict(X=P, W=P, t=1, N=2, V=100, D=64, ldx=64, ldw=64, ids=P, M=1, logp=P, m=P, s=P, ws=P, wb=BIG), **kw}
        return L.elmo_linear_logprobs(*(a[k] for k in "X W t N V D ldx ldw ids M logp m s ws wb".split()), None)
    for t in (0, 3, -1):
        assert call(t=t) == -3, t
    for bad in (dict(N=-1), dict(N=2**31), dict(V=0), dict(V=2**31), dict(D=0), dict(D=48), dict(D=65568, ldx=65568, ldw=65568), dict(ldx=63),
                dict(ldw=32), dict(ldx=1 << 22), dict(ldw=1 << 22), dict(M=65), dict(M=-1), dict(N=2**31 - 1, V=2**31 - 1),
                dict(N=1 << 21, V=1 << 21)):
        assert call(**bad) == -2, bad
    for bad in (dict(X=None), dict(W=None), dict(ids=None), dict(logp=None), dict(m=None), dict(s=None), dict(X=Q), dict(W=Q), dict(ldx=68),
                dict(ldw=68), dict(ids=ODD), dict(logp=Q), dict(m=ODD), dict(s=ODD)):
        assert call(**bad) == -1, bad
    for bad in (dict(ws=None), dict(ws=Q), dict(wb=8)):
        assert call(**bad) == -4, bad
    assert call(N=0, X=None) == 0
    f = L.elmo_linear_logprobs_workspace_bytes
    assert f(0, 100, 64, 1) == 0 and f(2, 100, 48, 1) == 0 and f(2, 100, 64, 65) == 0 and f(2, 0, 64, 1) == 0
    assert f(1, 1, 32, 0) > 0 and f(4096, 131072, 768, 1) < 4096 * 131072 // 8      # far from the logits' size


def test_linear_logprobs_backward(L):
    def call(**kw):
        a = {**dict(X=P, W=P, t=2, N=2, V=100, D=64, ldx=64, ldw=64, ids=P, M=1, m=P, s=P, g=P, gl=None, dX=O, xt=0, lddx=64, dW=O, wt=1, lddw=64,
                    acc=0, chunk=0, ws=P, wb=BIG), **kw}
        return L.elmo_linear_logprobs_backward(*(a[k] for k in "X W t N V D ldx ldw ids M m s g gl dX xt lddx dW wt lddw acc chunk ws wb".split()), None)
    for bad in (dict(t=0), dict(xt=3), dict(wt=-1)):
        assert call(**bad) == -3, bad
    for bad in (dict(N=-1), dict(V=0), dict(D=40), dict(ldx=63), dict(lddx=63), dict(lddw=63), dict(chunk=-1), dict(M=65)):
        assert call(**bad) == -2, bad
    for bad in (dict(dX=None, dW=None), dict(X=None), dict(W=None), dict(ids=None), dict(m=None), dict(s=None), dict(g=None), dict(dX=Q), dict(dW=Q),
                dict(lddx=66), dict(lddw=68), dict(X=Q), dict(gl=ODD), dict(g=Q)):
        assert call(**bad) == -1, bad
    for bad in (dict(ws=None), dict(ws=Q), dict(wb=8)):
        assert call(**bad) == -4, bad
    assert call(N=0, dW=None) == 0 and call(N=0, acc=1) == 0                        # nothing to do, nothing to add
    assert call(dX=None, xt=9, ws=None) == -4 and call(dW=None, wt=9, ws=None) == -4  # the type of what is not asked for
    f = L.elmo_linear_logprobs_backward_workspace_bytes
    assert f(0, 100, 64, 1, 0, 1, 1) == 0 and f(2, 100, 64, 1, -1, 1, 1) == 0 and f(2, 100, 40, 1, 0, 1, 1) == 0
    # a piece of 2^27 gradient codes at most, partial sums beside it; less with smaller pieces
    assert f(16384, 1 << 20, 768, 1, 0, 1, 1) < 2 * 2**27 + 64 * 16384 * 768 * 4
    assert f(5, 100, 64, 1, 2**63 - 1, 1, 1) == f(5, 100, 64, 1, 100, 1, 1)
    assert f(16384, 1 << 20, 768, 1, 1024, 1, 1) < f(16384, 1 << 20, 768, 1, 0, 1, 1)


def test_i8(L):
    def quant(**kw):
        a = {**dict(x=P, t=1, N=2, D=128, ld=128, c=P, s=P), **kw}
        return L.elmo_i8_quantize(*(a[k] for k in "x t N D ld c s".split()), None)
    assert quant(t=3) == -3
    for bad in (dict(N=-1), dict(N=2**31), dict(D=0), dict(D=96, ld=96), dict(D=65600, ld=65600), dict(ld=127)):
        assert quant(**bad) == -2, bad
    for bad in (dict(x=None), dict(c=None), dict(s=None), dict(x=Q), dict(c=Q), dict(ld=129), dict(s=ODD)):
        assert quant(**bad) == -1, bad
    assert quant(N=0, x=None) == 0

    def mul(**kw):
        a = {**dict(X=P, sx=P, W=P, sw=P, N=2, L=100, D=128, Y=P, t=0, ldy=100, ws=None, wb=0), **kw}
        return L.elmo_i8_matmul(*(a[k] for k in "X sx W sw N L D Y t ldy ws wb".split()), None)
    assert mul(t=3) == -3
    for bad in (dict(N=-1), dict(N=2**31), dict(L=0), dict(L=2**31), dict(D=32), dict(D=65600), dict(ldy=99), dict(N=2**31 - 1, L=2**31 - 1, ldy=2**31)):
        assert mul(**bad) == -2, bad
    for bad in (dict(X=None), dict(W=None), dict(sx=None), dict(sw=None), dict(Y=None), dict(X=Q), dict(W=Q), dict(sx=ODD), dict(sw=Q), dict(Y=Q)):
        assert mul(**bad) == -1, bad
    need = L.elmo_i8_matmul_workspace_bytes(40, 128, 65536)
    assert need >= 40 * 128 * 4 * 2
    for bad in (dict(), dict(ws=P, wb=need - 1), dict(ws=Q, wb=need)):
        assert mul(N=40, L=128, D=65536, ldy=128, **bad) == -4, bad
    assert mul(N=0, X=None) == 0
    assert L.elmo_i8_matmul_workspace_bytes(0, 100, 128) == 0 and L.elmo_i8_matmul_workspace_bytes(2, 100, 96) == 0


def test_dropout(L):
    def call(**kw):
        a = {**dict(x=P, t=0, T=4, D=8, ldx=8, r=None, ldr=0, p=0.5, seed=1, step=2, at=None, first=0, y=O, ldy=8), **kw}
        return L.elmo_dropout(*(a[k] for k in "x t T D ldx r ldr p seed step at first y ldy".split()), None)
    assert call(t=3) == -3
    for bad in (dict(T=-1), dict(T=2**31), dict(D=0), dict(D=2**31), dict(ldx=7), dict(ldy=7), dict(r=P, ldr=7), dict(y=P, ldy=9), dict(r=O, ldr=9)):
        assert call(**bad) == -2, bad
    for bad in (dict(p=-0.01), dict(p=1.01), dict(p=float("nan")), dict(first=2**64 - 31), dict(x=None), dict(y=None), dict(x=Q), dict(y=Q),
                dict(r=Q, ldr=8), dict(at=ctypes.c_void_p(4100))):
        assert call(**bad) == -1, bad
    assert call(T=0, x=None) == 0

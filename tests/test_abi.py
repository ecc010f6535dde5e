"""The C-ABI library loads and exports every entry point that include/elmo_xmc.h declares, and
rejects invalid arguments on the host (no GPU needed: validation happens before any HIP call)."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "elmo_xmc.h")


def declared_functions():
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(elmo_\w+)\s*\(", text)))


@pytest.fixture(scope="module")
def L():
    import precision_label_chunk_amd as elmo
    if not os.path.exists(elmo.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return elmo.lib()


def test_header_declares_the_boundary():
    names = declared_functions()
    for n in ["elmo_xmc_step", "elmo_xmc_topk", "elmo_xmc_step_workspace_bytes", "elmo_xmc_topk_workspace_bytes",
              "elmo_xmc_logits", "elmo_numerics_probe", "elmo_status_str", "elmo_abi_version", "elmo_xmc_step_flags",
              "elmo_kahan_update", "elmo_xmc_step_single_pass", "elmo_xmc_step_two_kernel"]:
        assert n in names


def test_library_exports_every_declared_symbol(L):
    for n in declared_functions():
        assert hasattr(L, n), f"missing export {n}"


def test_status_strings_and_version(L):
    assert L.elmo_abi_version() == 1
    assert L.elmo_status_str(0) == b"ok"
    assert L.elmo_status_str(-4).startswith(b"workspace")


@pytest.mark.parametrize("B,D,Lab,chunk,wd", [(0, 768, 1000, 128, 0), (257, 768, 1000, 128, 0), (4, 96, 1000, 128, 0),
                                              (4, 2048, 1000, 128, 0), (4, 768, 0, 128, 0), (4, 768, 1000, 0, 0),
                                              (4, 768, 1000, 128, 7), (4, 768, 2**31, 128, 0),
                                              (4, 192, 1000, 128, 2), (4, 640, 1000, 128, 2)])   # MXFP4: D % 256
def test_workspace_query_rejects_bad_shapes(L, B, D, Lab, chunk, wd):
    assert L.elmo_xmc_step_workspace_bytes(B, D, Lab, chunk, wd, 10) == 0


def test_step_rejects_invalid_arguments_before_launch(L):
    null = None
    # unknown format
    assert L.elmo_xmc_step(null, 5, 1000, 768, null, 4, null, null, 0, 0.1, 0, 0, 128, null, null, null, 0, null) == -3
    # bad shapes
    assert L.elmo_xmc_step(null, 0, 1000, 100, null, 4, null, null, 0, 0.1, 0, 0, 128, null, null, null, 0, null) == -2
    # null pointers
    assert L.elmo_xmc_step(null, 0, 1000, 128, null, 4, null, null, 0, 0.1, 0, 0, 128, null, null, null, 0, null) == -1
    # non-finite learning rate
    p = ctypes.c_void_p(4096)
    assert L.elmo_xmc_step(p, 0, 1000, 128, p, 4, p, p, 1, float("nan"), 0, 0, 128, p, null, p, 1 << 30, null) == -1
    # misaligned pointer
    q = ctypes.c_void_p(4097)
    assert L.elmo_xmc_step(q, 0, 1000, 128, p, 4, p, p, 1, 0.1, 0, 0, 128, p, null, p, 1 << 30, null) == -1
    # workspace too small (validation precedes any device work)
    assert L.elmo_xmc_step(p, 0, 1000, 128, p, 4, p, p, 1, 0.1, 0, 0, 128, p, null, p, 16, null) == -4
    # MXFP4 rows need D % 256 == 0
    assert L.elmo_xmc_step(p, 2, 1000, 192, p, 4, p, p, 1, 0.1, 0, 0, 128, p, null, p, 1 << 30, null) == -2
    assert L.elmo_xmc_step_workspace_bytes(4, 256, 1000, 128, 2, 10) > 0


def test_topk_rejects_invalid_arguments(L):
    null = None
    assert L.elmo_xmc_topk(null, 0, 1000, 128, null, 4, 0, null, null, null, 0, null) == -2
    assert L.elmo_xmc_topk(null, 0, 1000, 128, null, 4, 65, null, null, null, 0, null) == -2      # k > 64
    assert L.elmo_xmc_topk(null, 0, 10, 128, null, 4, 11, null, null, null, 0, null) == -2
    assert L.elmo_xmc_topk(null, 0, 1000, 128, null, 4, 5, null, null, null, 0, null) == -1
    assert L.elmo_xmc_topk_workspace_bytes(4, 128, 1000, 0, 0) == 0
    assert L.elmo_xmc_topk_workspace_bytes(4, 128, 1000, 5, 2) == 0       # MXFP4 with D % 256 != 0
    assert L.elmo_xmc_topk(null, 2, 1000, 128, null, 4, 5, null, null, null, 0, null) == -2


def test_numerics_probe_rejects_bad_op(L):
    assert L.elmo_numerics_probe(10, None, None, ctypes.c_void_p(4096), 1, 0, 0, None) == -1
    assert L.elmo_numerics_probe(8, ctypes.c_void_p(4096), None, ctypes.c_void_p(4096), 1, 0, 0, None) == -1
    assert L.elmo_numerics_probe(3, ctypes.c_void_p(4096), None, ctypes.c_void_p(4096), 1, 0, 0, None) == -1


def test_kahan_update_rejects_invalid_arguments(L):
    L.elmo_kahan_update.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                    ctypes.c_float, ctypes.c_void_p]
    p = ctypes.c_void_p(4096)
    assert L.elmo_kahan_update(p, p, p, -1, 0.1, None) == -2
    assert L.elmo_kahan_update(None, None, None, 0, 0.1, None) == 0          # empty: nothing to do
    assert L.elmo_kahan_update(None, p, p, 8, 0.1, None) == -1
    assert L.elmo_kahan_update(p, p, ctypes.c_void_p(4098), 8, 0.1, None) == -1   # misaligned g
    assert L.elmo_kahan_update(ctypes.c_void_p(4097), p, p, 8, 0.1, None) == -1   # misaligned w


def test_single_pass_step_rejects_shapes_it_does_not_build(L):
    null = None
    p = ctypes.c_void_p(4096)
    f = L.elmo_xmc_step_single_pass
    f.restype = ctypes.c_int
    # the same host validation as elmo_xmc_step
    assert f(null, 5, 1000, 768, null, 4, null, null, 0, 0.1, 0, 0, 128, null, null, null, null, 0, null) == -3
    assert f(null, 0, 1000, 100, null, 4, null, null, 0, 0.1, 0, 0, 128, null, null, null, null, 0, null) == -2
    assert f(p, 0, 1000, 768, p, 4, p, p, 1, float("nan"), 0, 0, 128, p, null, null, p, 1 << 30, null) == -1
    # built for B <= 32 and D in {256, 512, 768} only: other valid shapes are unsupported, nothing runs
    assert f(p, 0, 1000, 768, p, 33, p, p, 1, 0.1, 0, 0, 128, p, null, null, p, 1 << 30, null) == -6
    assert f(p, 1, 1000, 640, p, 8, p, p, 1, 0.1, 0, 0, 128, p, null, null, p, 1 << 30, null) == -6
    assert f(p, 0, 1000, 1024, p, 8, p, p, 1, 0.1, 0, 0, 128, p, null, null, p, 1 << 30, null) == -6
    # workspace too small for a supported shape; a misaligned gradient-code output
    assert f(p, 0, 1000, 768, p, 32, p, p, 1, 0.1, 0, 0, 128, p, null, null, p, 16, null) == -4
    assert f(p, 0, 1000, 768, p, 32, p, p, 1, 0.1, 0, 0, 128, p, null, ctypes.c_void_p(4097), p, 1 << 30,
             null) == -1


def test_workspace_holds_the_single_pass_partials():
    """At padded batch 32 and D = 768 the workspace has room for one dX partial (32 x 768 FP32) per
    single-pass work-group, up to one per CU (or per 32-label tile of the chunk, if fewer)."""
    import precision_label_chunk_amd as elmo
    small = elmo.step_workspace_bytes(32, 768, 4096, 1024, 0, 100)
    big = elmo.step_workspace_bytes(32, 768, 8_600_000, 262_144, 0, 100)
    assert small >= 32 * (32 * 768 * 4)
    assert big >= 256 * (32 * 768 * 4)


def test_two_kernel_step_validates_like_the_step(L):
    null = None
    p = ctypes.c_void_p(4096)
    f = L.elmo_xmc_step_two_kernel
    assert f(null, 5, 1000, 768, null, 4, null, null, 0, 0.1, 0, 0, 128, null, null, null, 0, null) == -3
    assert f(null, 0, 1000, 100, null, 4, null, null, 0, 0.1, 0, 0, 128, null, null, null, 0, null) == -2
    assert f(p, 0, 1000, 768, p, 4, p, p, 1, float("nan"), 0, 0, 128, p, null, p, 1 << 30, null) == -1
    assert f(p, 0, 1000, 768, p, 32, p, p, 1, 0.1, 0, 0, 128, p, null, p, 16, null) == -4


def test_logprobs_rejects_invalid_arguments(L):
    p, q, w = ctypes.c_void_p(4096), ctypes.c_void_p(4097), 1 << 30
    f = L.elmo_logprobs
    ok = dict(Z=p, t=0, N=2, V=100, ld=100, ids=p, M=1, k=5, logp=p, H=p, m=p, s=p, ti=p, tl=p, ws=p, wb=w)

    def call(**kw):
        a = {**ok, **kw}
        return f(a["Z"], a["t"], a["N"], a["V"], a["ld"], a["ids"], a["M"], a["k"], a["logp"], a["H"], a["m"], a["s"],
                 a["ti"], a["tl"], a["ws"], a["wb"], None)
    assert call(t=3) == -3
    for bad in (dict(N=-1), dict(N=2**31), dict(V=0), dict(V=2**31), dict(ld=99), dict(M=65), dict(M=-1), dict(k=65),
                dict(k=-1), dict(V=4, ld=4, k=5)):
        assert call(**bad) == -2, bad
    for bad in (dict(Z=None), dict(ids=None), dict(logp=None), dict(H=None), dict(m=None), dict(s=None), dict(ti=None),
                dict(tl=None), dict(Z=q), dict(ids=ctypes.c_void_p(4098)), dict(tl=q)):
        assert call(**bad) == -1, bad
    for bad in (dict(ws=None), dict(ws=q), dict(wb=8)):
        assert call(**bad) == -4, bad
    assert call(N=0, Z=None) == 0
    assert L.elmo_logprobs_workspace_bytes(2, 100, 101) == 0 and L.elmo_logprobs_workspace_bytes(0, 100, 1) == 0
    assert L.elmo_logprobs_workspace_bytes(1, 1 << 20, 64) >= 64 * 8
    g = L.elmo_logprobs_backward

    def grad(**kw):
        a = {**dict(Z=p, t=1, N=2, V=100, ld=100, ids=p, M=1, m=p, s=p, H=p, g=p, gH=None, gL=None,
                    d=ctypes.c_void_p(8192), ldd=100), **kw}
        return g(a["Z"], a["t"], a["N"], a["V"], a["ld"], a["ids"], a["M"], a["m"], a["s"], a["H"], a["g"], a["gH"],
                 a["gL"], a["d"], a["ldd"], None)
    assert grad(t=-1) == -3
    assert grad(ldd=99) == -2 and grad(d=p, ldd=101) == -2 and grad(M=65) == -2
    for bad in (dict(Z=None), dict(d=None), dict(m=None), dict(s=None), dict(H=None), dict(g=None), dict(ids=None),
                dict(d=q), dict(gH=q), dict(gL=q)):
        assert grad(**bad) == -1, bad
    assert grad(N=0) == 0


def test_w4_matvec_rejects_invalid_arguments(L):
    p, q = ctypes.c_void_p(4096), ctypes.c_void_p(4097)

    def mx(**kw):
        a = {**dict(W=p, f=2, L=10, D=256, G=32, s=None, z=None, X=p, N=2, ldx=256, Y=p, t=0, ldy=10), **kw}
        return L.elmo_w4_matvec(a["W"], a["f"], a["L"], a["D"], a["G"], a["s"], a["z"], a["X"], a["N"], a["ldx"], a["Y"],
                                a["t"], a["ldy"], None)

    def i4(**kw):
        return mx(**{**dict(f=3, G=64, s=p), **kw})
    assert mx(f=1) == -3 and mx(f=4) == -3 and mx(t=3) == -3
    for bad in (dict(N=33), dict(N=-1), dict(L=0), dict(L=2**31), dict(D=0), dict(D=128, ldx=128), dict(D=65792, ldx=65792),
                dict(G=64), dict(ldx=248), dict(ldx=260), dict(ldy=9)):
        assert mx(**bad) == -2, bad
    for bad in (dict(G=16), dict(G=256), dict(D=224, ldx=256), dict(G=128, D=192)):
        assert i4(**bad) == -2, bad
    for bad in (dict(W=None), dict(X=None), dict(Y=None), dict(W=ctypes.c_void_p(4100)), dict(X=ctypes.c_void_p(4104)),
                dict(Y=ctypes.c_void_p(4098)), dict(s=p), dict(z=p)):
        assert mx(**bad) == -1, bad
    for bad in (dict(s=None), dict(s=q), dict(W=ctypes.c_void_p(4104))):
        assert i4(**bad) == -1, bad
    assert mx(N=0, W=None) == 0


def test_ckpt8_rejects_invalid_arguments(L):
    p, q, o = ctypes.c_void_p(4096), ctypes.c_void_p(4100), ctypes.c_void_p(65536)

    def save(**kw):
        a = {**dict(x=p, t=1, T=2, D=64, ld=64, act=3, c=p, s=p, y=o, ldy=64), **kw}
        return L.elmo_ckpt8_save(a["x"], a["t"], a["T"], a["D"], a["ld"], a["act"], a["c"], a["s"], a["y"], a["ldy"], None)
    assert save(t=3) == -3
    for bad in (dict(T=-1), dict(D=0), dict(D=48, ld=48), dict(ld=63), dict(ldy=32), dict(T=2**31)):
        assert save(**bad) == -2, bad
    for bad in (dict(x=None), dict(c=None), dict(s=None), dict(act=4), dict(act=-1), dict(act=0), dict(y=None), dict(x=q),
                dict(c=q), dict(ld=68), dict(y=q), dict(ldy=68)):
        assert save(**bad) == -1, bad
    assert save(T=0, x=None) == 0
    assert L.elmo_ckpt8_load(p, p, 2, 48, p, 1, 48, None) == -2 and L.elmo_ckpt8_load(None, p, 2, 64, p, 1, 64, None) == -1
    assert L.elmo_ckpt8_load(p, p, 2, 64, p, 1, 68, None) == -1 and L.elmo_ckpt8_load(p, p, 2, 64, p, 7, 64, None) == -3

    def grad(**kw):
        a = {**dict(dy=p, t=1, T=2, D=64, ld=64, act=1, c=p, s=p, dx=o, ldx=64), **kw}
        return L.elmo_ckpt8_act_grad(a["dy"], a["t"], a["T"], a["D"], a["ld"], a["act"], a["c"], a["s"], a["dx"], a["ldx"], None)
    assert grad(t=9) == -3 and grad(D=33) == -2 and grad(ldx=63) == -2 and grad(dx=p, ldx=72) == -2
    for bad in (dict(act=0), dict(act=4), dict(dy=None), dict(dx=None), dict(c=None), dict(s=None), dict(dx=q), dict(ld=68)):
        assert grad(**bad) == -1, bad

    def wgrad(**kw):
        a = {**dict(dy=p, ldy=16, c=p, s=p, T=4, O=16, D=64, dW=o, acc=0, ws=p, wb=1 << 30), **kw}
        return L.elmo_ckpt8_weight_grad(a["dy"], a["ldy"], a["c"], a["s"], a["T"], a["O"], a["D"], a["dW"], a["acc"],
                                        a["ws"], a["wb"], None)
    for bad in (dict(O=0), dict(O=12), dict(D=40), dict(T=-1), dict(ldy=8), dict(ldy=20)):
        assert wgrad(**bad) == -2, bad
    for bad in (dict(dy=None), dict(c=None), dict(s=None), dict(dW=None), dict(dW=q), dict(dy=q), dict(c=q)):
        assert wgrad(**bad) == -1, bad
    for bad in (dict(ws=None), dict(ws=q), dict(wb=1)):
        assert wgrad(**bad) == -4, bad
    assert L.elmo_ckpt8_weight_grad_workspace_bytes(4, 12, 64) == 0
    assert L.elmo_ckpt8_weight_grad_workspace_bytes(1 << 20, 768, 768) >= 768 * 768 * 4

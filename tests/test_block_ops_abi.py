"""CPU-only checks of the C entry points of the feed-forward block: arguments
are refused on the host, before any launch, and sizes of workspaces."""
import ctypes
import os

import pytest

from fp8_block_scaled_04_amd import binding as b, build

OK, EINVAL, EUNSUPPORTED = b.FP8G_OK, b.FP8G_EINVAL, b.FP8G_EUNSUPPORTED
P = ctypes.c_void_p(0x1000)      # an aligned address that is never read
Q = ctypes.c_void_p(0x2000)
ODD = ctypes.c_void_p(0x1008)    # not 16-byte aligned


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(build.LIB):
        build.build()
    return b.lib()


def _call(fn, args, **over):
    return fn(*{**args, **over}.values())


def _refusals(fn, args, einval=(), eunsupported=(), ok=()):
    for over in einval:
        assert _call(fn, args, **over) == EINVAL, over
    for over in eunsupported:
        assert _call(fn, args, **over) == EUNSUPPORTED, over
    for over in ok:
        assert _call(fn, args, **over) == OK, over


def test_gemm_epilogue_refusals(lib):
    a = dict(lhs=P, lf=0, ls=P, ld=16, rhs=P, rf=0, rs=P, bias=P, bd=0, act=0, residual=P, preact=Q, out=P, m=16, n=64,
             k=256, ws=None, wb=0, stream=None)
    _refusals(lib.fp8_gemm_nt_epilogue, a,
              einval=[dict(lhs=None), dict(ls=None), dict(rhs=None), dict(rs=None), dict(out=None), dict(lf=2),
                      dict(rf=-1), dict(bd=2), dict(act=-1), dict(act=5), dict(m=-1), dict(n=-8), dict(bias=ODD),
                      dict(residual=ODD), dict(preact=ODD), dict(out=ODD), dict(lhs=ODD), dict(ws=ODD, wb=1 << 20),
                      dict(preact=P), dict(out=Q, residual=P, preact=Q), dict(residual=Q, preact=Q)],
              eunsupported=[dict(n=12), dict(k=100), dict(k=0), dict(k=65664), dict(ld=15), dict(ld=12)],
              ok=[dict(m=0), dict(n=0), dict(m=0, lhs=None)])


def test_epilogue_backward_refusals(lib):
    a = dict(go=P, z=P, act=4, m=100, n=64, gz=P, gb=P, ws=P, wb=1 << 20, stream=None)
    assert lib.fp8_epilogue_backward_workspace_bytes(100, 64) > 0
    _refusals(lib.fp8_epilogue_backward, a,
              einval=[dict(go=None), dict(z=None), dict(gz=None), dict(act=5), dict(act=-1), dict(m=-1), dict(n=-8),
                      dict(go=ODD), dict(z=ODD), dict(gz=ODD), dict(gb=ODD), dict(ws=ODD), dict(ws=None),
                      dict(wb=16)],
              eunsupported=[dict(n=12)], ok=[dict(n=0), dict(m=0, gb=None)])


def test_norm_refusals(lib):
    a = dict(x=P, xd=1, xld=64, r=P, rld=64, sd=1, T=4, n=64, kind=0, eps=1e-6, post=1, pw=P, gate=P, grows=1, scale=1.0,
             prew=P, pd=0, h=P, y=P, q=P, qf=0, qs=P, qld=4, stream=None)
    _refusals(lib.fp8_norm_residual, a,
              einval=[dict(x=None), dict(xd=2), dict(sd=2), dict(pd=3), dict(kind=2), dict(kind=-1), dict(T=-1),
                      dict(n=-8), dict(xld=56), dict(rld=56), dict(grows=2), dict(grows=0), dict(eps=-1.0),
                      dict(eps=float("nan")), dict(h=None, y=None, q=None), dict(qs=None), dict(qf=2), dict(x=ODD),
                      dict(r=ODD), dict(pw=ODD), dict(gate=ODD), dict(prew=ODD), dict(h=ODD), dict(y=ODD), dict(q=ODD),
                      dict(qs=ODD)],
              eunsupported=[dict(n=60), dict(n=16392, xld=16392, rld=16392), dict(xld=68), dict(rld=68), dict(qld=3)],
              ok=[dict(T=0), dict(n=0), dict(T=0, x=None)])


def test_norm_backward_refusals(lib):
    a = dict(gh=P, gy=P, x=P, xd=1, xld=64, h=P, sd=1, T=4, n=64, kind=1, eps=1e-6, post=1, pw=P, gate=P, grows=1,
             scale=1.0, prew=P, pd=0, gx=P, gr=P, gpre=P, gpost=P, ggate=P, ws=P, wb=1 << 20, stream=None)
    needed = lib.fp8_norm_residual_backward_workspace_bytes(4, 64)
    assert 0 < needed <= 4 * 3 * 64 * 4
    _refusals(lib.fp8_norm_residual_backward, a,
              einval=[dict(gh=None, gy=None, gpre=None), dict(x=None), dict(h=None), dict(xd=2), dict(sd=-1), dict(pd=2),
                      dict(kind=2), dict(T=-1), dict(n=-8), dict(xld=56), dict(grows=3), dict(eps=-1.0), dict(ws=None),
                      dict(wb=needed - 1), dict(post=0), dict(gate=None), dict(gy=None),
                      dict(gx=None, gr=None, gpre=None, gpost=None, ggate=None), dict(gh=ODD), dict(gy=ODD), dict(x=ODD),
                      dict(h=ODD), dict(pw=ODD), dict(gate=ODD), dict(prew=ODD), dict(gx=ODD), dict(gr=ODD),
                      dict(gpre=ODD), dict(gpost=ODD), dict(ggate=ODD), dict(ws=ODD)],
              eunsupported=[dict(n=60), dict(n=16392, xld=16392), dict(xld=68)],
              ok=[dict(n=0), dict(T=0, gpre=None, gpost=None, ggate=None)])


def test_moe_few_tokens_refusals(lib):
    a = dict(x=P, xld=256, idx=P, w=P, T=4, topk=2, up=P, us=P, down=P, ds=P, E=8, hidden=256, inter=128, act=4, out=P,
             ws=P, wb=1 << 24, stream=None)
    needed = lib.fp8_moe_few_tokens_workspace_bytes(4, 2, 256, 128)
    _refusals(lib.fp8_moe_few_tokens, a,
              einval=[dict(x=None), dict(idx=None), dict(up=None), dict(us=None), dict(down=None), dict(ds=None),
                      dict(out=None), dict(ws=None), dict(wb=needed - 1), dict(T=-1), dict(topk=0), dict(E=0),
                      dict(hidden=-128), dict(inter=-128), dict(act=5), dict(act=-1), dict(xld=248), dict(x=ODD),
                      dict(up=ODD), dict(us=ODD), dict(down=ODD), dict(ds=ODD), dict(out=ODD), dict(ws=ODD),
                      dict(idx=ctypes.c_void_p(0x1002)), dict(w=ctypes.c_void_p(0x1002))],
              eunsupported=[dict(topk=33), dict(E=4097), dict(hidden=192), dict(inter=64), dict(inter=0),
                            dict(hidden=65664, xld=65664), dict(inter=65664), dict(xld=260)],
              ok=[dict(T=0), dict(hidden=0, xld=0)])


def test_workspace_sizes(lib):
    w = lib.fp8_moe_few_tokens_workspace_bytes
    assert w(0, 8, 1024, 512) == 0 and w(4, 0, 1024, 512) == 0 and w(4, 33, 1024, 512) == 0
    # a launch takes at most 64 tokens and 512 pairs, so more tokens need no more
    assert w(64, 8, 1024, 512) == w(1000, 8, 1024, 512) > w(3, 8, 1024, 512) > 3 * 8 * 512 * 2
    assert lib.fp8_epilogue_backward_workspace_bytes(16, 1024) == 0       # one slice
    assert lib.fp8_epilogue_backward_workspace_bytes(0, 8) == 0
    assert lib.fp8_norm_residual_backward_workspace_bytes(0, 8) == 0
    # 512 slices at most
    assert lib.fp8_norm_residual_backward_workspace_bytes(1 << 20, 1024) == 512 * 3 * 1024 * 4


def test_sizes_past_32_bit_rows_and_grids_are_refused(lib):
    """Row numbers and grids are 32 bits: nothing near their end reaches a kernel."""
    past = (1 << 30) + 1
    assert lib.fp8_epilogue_backward(P, P, 4, past, 64, P, None, None, 0, None) == EUNSUPPORTED
    assert lib.fp8_epilogue_backward(P, P, 4, 1, 1 << 28, P, None, None, 0, None) == EUNSUPPORTED
    for rows, n in ((past, 8), (2 ** 31 - 1, 8), (1 << 22, 1024), (1 << 24, 512)):
        assert lib.fp8_norm_residual(P, 1, n, None, n, 1, rows, n, 0, 1e-6, 0, None, None, 1, 1.0, None, 0, P, None, None,
                                     0, None, rows, None) == EUNSUPPORTED, (rows, n)
    for rows in (past, 2 ** 31 - 1):
        assert lib.fp8_norm_residual_backward(P, None, None, 1, 8, None, 1, rows, 8, 0, 1e-6, 0, None, None, 1, 1.0, None,
                                              0, P, None, None, None, None, None, 0, None) == EUNSUPPORTED


def test_norm_backward_asks_nothing_of_an_absent_x(lib):
    """Without x its row stride is not looked at (no rows: nothing is launched)."""
    args = (P, P, None, 1, 0, P, 1, 0, 64, 0, 1e-6, 0, None, None, 1, 1.0, None, 0, P, P, None, None, None, None, 0, None)
    assert lib.fp8_norm_residual_backward(*args) == OK

"""Host-side refusals of the norm, the quantised-row permutation and the few-token layer: an
invalid call returns its status before anything is launched (no GPU needed)."""
import ctypes as C

import pytest

import __graft_entry__
from mixture_experts_ffn_warp_gb300 import _binding

INF, NAN = float("inf"), float("nan")
P, MIS, NUL = C.c_void_p(16), C.c_void_p(24), None
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 5


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return _binding.load_library()


def norm(lib, x=P, res=P, w=P, eps=1e-6, T=4, H=64, sum=P, y=P, yq=NUL, ysf=NUL, rstd=P):
    return lib.moe_add_rmsnorm(x, res, w, eps, T, H, sum, y, yq, ysf, rstd, NUL)


def test_norm_refusals(lib):
    assert norm(lib, T=0) == OK
    assert norm(lib, x=NUL) == INVALID
    assert norm(lib, w=NUL) == INVALID
    assert norm(lib, y=NUL) == INVALID                     # no output wanted
    assert norm(lib, yq=P) == INVALID                      # codes without scales
    assert norm(lib, ysf=P) == INVALID
    assert norm(lib, sum=NUL) == INVALID                   # residual without its sum
    assert norm(lib, eps=-1.0) == INVALID and norm(lib, eps=NAN) == INVALID
    assert norm(lib, T=-1) == INVALID and norm(lib, H=0) == INVALID
    assert norm(lib, H=60) == UNSUPPORTED                  # H % 8
    assert norm(lib, H=40, yq=P, ysf=P) == UNSUPPORTED     # H % 32 with MXFP8
    assert norm(lib, H=32776) == UNSUPPORTED
    assert norm(lib, T=1 << 31) == UNSUPPORTED
    for name in ("x", "res", "w", "sum", "y"):
        assert norm(lib, **{name: MIS}) == UNSUPPORTED, name
    assert norm(lib, yq=C.c_void_p(20), ysf=P) == UNSUPPORTED


def test_norm_bwd_refusals(lib):
    need = lib.moe_rmsnorm_bwd_workspace_bytes(4, 64)
    assert need > 0
    assert lib.moe_rmsnorm_bwd_workspace_bytes(4, 60) == 0 and lib.moe_rmsnorm_bwd_workspace_bytes(-1, 64) == 0
    # more rows never need less
    sizes = [lib.moe_rmsnorm_bwd_workspace_bytes(t, 4096) for t in (0, 1, 10, 300, 1000, 100000)]
    assert sizes == sorted(sizes)

    def bwd(dy=P, ds=P, s=P, w=P, rstd=P, T=4, H=64, dx=P, dw=P, ws=P, n=need):
        return lib.moe_add_rmsnorm_bwd(dy, ds, s, w, rstd, T, H, dx, dw, ws, n, NUL)
    assert bwd(T=0, dw=NUL) == OK
    for name in ("dy", "s", "w", "rstd", "dx"):
        assert bwd(**{name: NUL}) == INVALID, name
    assert bwd(ws=NUL) == WORKSPACE and bwd(n=need - 1) == WORKSPACE
    assert bwd(H=60) == UNSUPPORTED and bwd(T=-1) == INVALID
    for name in ("dy", "ds", "s", "w", "dx", "ws"):
        assert bwd(**{name: MIS}) == UNSUPPORTED, name


def test_permute_rows_refusals(lib):
    def perm(q=P, sf=P, idx=P, T=4, H=128, E=4, k=2, xq=P, xsf=P, cap=8, dst=P, src=P, gs=P, go=P, ws=NUL, n=0):
        return lib.moe_permute_rows_mxfp8(q, sf, idx, T, H, E, k, xq, xsf, cap, dst, src, gs, go, ws, n, NUL)
    assert perm() == WORKSPACE
    assert perm(H=64) == UNSUPPORTED and perm(E=1025) == UNSUPPORTED and perm(k=33) == UNSUPPORTED
    assert perm(cap=7) == INVALID and perm(T=-1) == INVALID
    for name in ("q", "sf", "idx", "xq", "xsf", "dst", "src", "gs", "go"):
        assert perm(**{name: NUL}) == INVALID, name
    assert perm(q=MIS) == UNSUPPORTED and perm(xq=MIS) == UNSUPPORTED
    assert perm(sf=C.c_void_p(18)) == UNSUPPORTED and perm(xsf=C.c_void_p(18)) == UNSUPPORTED


@pytest.mark.parametrize("mx", [False, True])
def test_decode_refusals(lib, mx):
    W = 6 if mx else 3
    fn = lib.moe_decode_mxfp8 if mx else lib.moe_decode

    def dec(x=P, lg=P, bias=NUL, score=0, clamp=(-INF, INF, -INF, INF), w=None, T=2, H=128, F=256, E=8, k=2, idx=P,
            tw=P, out=P, ws=P, n=1 << 40):
        return fn(x, lg, bias, score, 1, *clamp, *(w or [P] * W), T, H, F, E, k, idx, tw, out, ws, n, NUL)
    assert dec(T=0) == OK
    assert dec(T=-1) == INVALID and dec(score=2) == INVALID
    for name in ("x", "lg", "idx", "tw", "out"):
        assert dec(**{name: NUL}) == INVALID, name
    for i in range(W):
        assert dec(w=[NUL if j == i else P for j in range(W)]) == INVALID
        assert dec(w=[MIS if j == i else P for j in range(W)]) == UNSUPPORTED
    assert dec(clamp=(1.0, 0.5, -INF, INF)) == INVALID and dec(clamp=(-INF, INF, NAN, 1.0)) == INVALID
    assert dec(T=65) == UNSUPPORTED
    assert dec(H=192) == UNSUPPORTED and dec(F=64) == UNSUPPORTED
    assert dec(E=1025) == UNSUPPORTED and dec(k=9) == UNSUPPORTED and dec(E=64, k=33) == UNSUPPORTED
    assert dec(x=MIS) == UNSUPPORTED and dec(out=MIS) == UNSUPPORTED
    need = lib.moe_decode_workspace_bytes(2, 128, 256, 8, 2)
    assert dec(ws=NUL) == WORKSPACE and dec(n=need - 1) == WORKSPACE


def test_decode_workspace_bytes(lib):
    f = lib.moe_decode_workspace_bytes
    assert f(1, 128, 256, 8, 2) >= 256
    assert f(65, 128, 256, 8, 2) == 0 and f(1, 100, 256, 8, 2) == 0 and f(1, 128, 256, 8, 9) == 0
    assert f(1, 128, 256, 2000, 2) == 0 and f(-1, 128, 256, 8, 2) == 0
    sizes = [f(t, 2048, 1408, 64, 6) for t in range(0, 65)]   # a workspace for T serves fewer tokens
    assert sizes == sorted(sizes)
    assert lib.moe_decode_workspace_init(NUL, 4096, NUL) == WORKSPACE
    assert lib.moe_decode_workspace_init(P, 8, NUL) == WORKSPACE

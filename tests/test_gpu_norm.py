"""moe_add_rmsnorm / moe_add_rmsnorm_bwd against the formulas in 64 bits, the gradient also
against differences, and moe_permute_rows_mxfp8 against the quantising permutation.

Bounds.  A correctly rounded output differs from the exact value by at most half a step of
its format; the fp32 arithmetic in front of that rounding adds a relative error of the sum of
squares (at most 128 sequential additions a thread and 8 + 5 levels of tree: 141 * 2^-24, half
of it in rstd) and a handful of roundings, below REL = 1e-5 together."""
import numpy as np
import pytest
import torch

import oracle
from helpers import bf16_half_ulp, e4m3_half_step, to_f64
from mixture_experts_ffn_warp_gb300 import (MoeForwardMX, MxWeights, NormOutput, NormWorkspace, PermutationMX,
                                            Workspace, moe_add_rmsnorm, moe_add_rmsnorm_bwd,
                                            moe_grouped_quantize_mxfp8, moe_permute_mxfp8, moe_permute_rows_mxfp8,
                                            moe_route_topk)
from mixture_experts_ffn_warp_gb300._binding import MoeError

pytestmark = pytest.mark.gpu
REL = 1e-5
EPS = 1e-6


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def inputs(T, H, seed=0, residual=True, scale=1.0):
    g = gen(seed)
    x = (torch.randn(T, H, generator=g, device="cuda") * scale).to(torch.bfloat16)
    r = (3 * torch.randn(T, H, generator=g, device="cuda") * scale).to(torch.bfloat16) if residual else None
    w = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
    return x, r, w


def reference(x, r, w, eps=EPS):
    s = to_f64(x) + (to_f64(r) if r is not None else 0.0)
    rstd = 1.0 / np.sqrt((s ** 2).mean(-1) + eps)
    return s, rstd, s * rstd[:, None] * to_f64(w)


def check_bf16(got, ref, what, extra=0.0):
    bound = bf16_half_ulp(ref) + REL * np.abs(ref) + extra
    bad = ~(np.abs(to_f64(got) - ref) <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3])


SHAPES = [(1, 8), (1, 128), (2, 4096), (3, 2048), (7, 2056), (5, 4104), (64, 7168), (33, 8192), (4, 16392), (2, 32768),
          (1000, 136)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("residual", [True, False])
def test_forward_bf16(T, H, residual):
    x, r, w = inputs(T, H, seed=T + H, residual=residual)
    o = moe_add_rmsnorm(x, w, EPS, residual=r)
    s, rstd, y = reference(x, r, w)
    assert (o.sum is not None) == residual
    if residual:
        check_bf16(o.sum, s, "sum")
    np.testing.assert_allclose(to_f64(o.rstd), rstd, rtol=REL)
    check_bf16(o.y, y, "y")


@pytest.mark.parametrize("T,H", [(1, 32), (1, 4096), (5, 96), (3, 2080), (17, 7168), (2, 32768), (300, 1408)])
@pytest.mark.parametrize("bf16", [True, False])
def test_forward_mxfp8(T, H, bf16):
    x, r, w = inputs(T, H, seed=3 * T + H)
    o = moe_add_rmsnorm(x, w, EPS, residual=r, bf16=bf16, mxfp8=True)
    s, rstd, y = reference(x, r, w)
    check_bf16(o.sum, s, "sum")
    if bf16:
        check_bf16(o.y, y, "y")
    else:
        assert o.y is None
    amax = np.abs(y.reshape(T, H // 32, 32)).max(-1)
    # the smallest 2^X with amax <= 448 * 2^X; a maximum within REL of a threshold may go either way
    lo = np.ceil(np.log2(amax * (1 - REL) / 448.0)).astype(int) + 127
    hi = np.ceil(np.log2(amax * (1 + REL) / 448.0)).astype(int) + 127
    sf = o.y_sf.cpu().numpy().astype(int)
    assert ((sf == lo) | (sf == hi)).all()
    codes = np.vectorize(oracle.e4m3_to_double)(np.arange(256, dtype=np.uint8))[o.y_q.cpu().numpy()]
    val = codes * np.ldexp(1.0, np.repeat(sf - 127, 32, axis=-1))
    assert (np.abs(val - y) <= e4m3_half_step(y, sf) + REL * np.abs(y)).all()


def test_forward_special_rows():
    """A row of zeros gives zeros (scale byte 0), tiny and huge rows keep their scale, and a row with
    an infinity or a NaN stays alone in it."""
    T, H = 7, 256
    x, r, w = inputs(T, H, seed=5)
    x[0], r[0] = 0, 0
    x[1], r[1] = x[1] * 1e-20, 0
    x[2], r[2] = x[2] * 1e15, 0
    x[3, 5] = float("inf")
    x[4, 200] = float("nan")
    o = moe_add_rmsnorm(x, w, EPS, residual=r, bf16=True, mxfp8=True)
    y = to_f64(o.y)
    assert (y[0] == 0).all() and (o.y_q[0] & 0x7F == 0).all() and (o.y_sf[0] == 0).all()
    assert abs(float(o.rstd[0]) - 1e3) < 1e-2
    fine = [0, 1, 2, 5, 6]
    s, rstd, ref = reference(x, r, w)
    check_bf16(o.y[fine], ref[fine], "y")
    np.testing.assert_allclose(to_f64(o.rstd)[fine], rstd[fine], rtol=REL)
    assert np.isnan(y[3, 5]) and (y[3, :5] == 0).all()
    assert np.isnan(y[4]).all()


def test_forward_in_place_and_buffers():
    """sum written over the residual, and over x; buffers of a NormOutput are the ones written."""
    T, H = 9, 1024
    x, r, w = inputs(T, H, seed=8)
    a = moe_add_rmsnorm(x, w, EPS, residual=r, mxfp8=True)
    buf = NormOutput.empty(T, H, bf16=True, mxfp8=True)
    for over in ("residual", "x"):
        x2, r2 = x.clone(), r.clone()
        buf.sum = r2 if over == "residual" else x2
        b = moe_add_rmsnorm(x2, w, EPS, residual=r2, out=buf)
        assert b is buf
        for n in ("sum", "y", "y_q", "y_sf", "rstd"):
            assert torch.equal(getattr(a, n), getattr(b, n)), (over, n)


def test_zero_rows():
    H = 64
    x, r, w = inputs(0, H)
    o = moe_add_rmsnorm(x, w, EPS, residual=r)
    assert o.y.shape == (0, H)
    dw = torch.full((H,), 7.0, device="cuda")
    dx, dw = moe_add_rmsnorm_bwd(x, x, w, torch.empty(0, device="cuda"), dweight=dw)
    assert dx.shape == (0, H) and (dw == 0).all()


def bwd_reference(dy, s, w, rstd, ds):
    dy, s, w, rstd = to_f64(dy), to_f64(s), to_f64(w), to_f64(rstd)[:, None]
    xh = s * rstd
    g = dy * w
    m = (g * xh).mean(-1, keepdims=True)
    dx = rstd * (g - xh * m) + (to_f64(ds) if ds is not None else 0.0)
    # magnitudes that the fp32 roundings are relative to
    mag = rstd * (np.abs(g) + np.abs(xh) * np.abs(g * xh).mean(-1, keepdims=True)) + np.abs(dx)
    return dx, (dy * xh).sum(0), mag, np.abs(dy * xh).sum(0)


@pytest.mark.parametrize("T,H", [(1, 8), (1, 4096), (2, 136), (33, 2048), (333, 2056), (700, 512), (1300, 4104),
                                 (5, 8200), (3, 32768), (4096, 128), (400, 1600), (401, 1608), (400, 1592), (33, 136),
                                 (17, 72), (100, 7168), (399, 16384)])
@pytest.mark.parametrize("with_sum", [True, False])
def test_backward(T, H, with_sum):
    x, r, w = inputs(T, H, seed=T + 2 * H)
    o = moe_add_rmsnorm(x, w, EPS, residual=r)
    g = gen(T + 7)
    dy = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    ds = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16) if with_sum else None
    dx, dw = moe_add_rmsnorm_bwd(dy, o.sum, w, o.rstd, d_sum=ds)
    rx, rw, mag, wmag = bwd_reference(dy, o.sum, w, o.rstd, ds)
    # the mean's terms: at most 128 sequential additions a thread and the tree, as the forward's
    check_bf16(dx, rx, "dx", extra=REL * mag)
    # dw: T terms of three roundings, summed in fp32
    assert (np.abs(to_f64(dw) - rw) <= (T + 4) * 2.0 ** -24 * wmag).all()
    again = moe_add_rmsnorm_bwd(dy, o.sum, w, o.rstd, d_sum=ds, ws=NormWorkspace(T + 50, H))
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)     # the same bits
    only_x, none = moe_add_rmsnorm_bwd(dy, o.sum, w, o.rstd, d_sum=ds, want_dweight=False)
    assert none is None and torch.equal(only_x, dx)
    for over in ("dy", "d_sum") if with_sum else ("dy",):
        dy2, ds2 = dy.clone(), ds.clone() if with_sum else None
        got, dw2 = moe_add_rmsnorm_bwd(dy2, o.sum, w, o.rstd, d_sum=ds2, dx=dy2 if over == "dy" else ds2)
        assert torch.equal(got, dx), over
        assert (np.abs(to_f64(dw2) - rw) <= (T + 4) * 2.0 ** -24 * wmag).all(), over


def test_backward_against_differences():
    """The 64-bit gradient formula used above, against central differences of the forward's formula."""
    rng = np.random.default_rng(0)
    T, H = 3, 24
    s, w, dy = rng.normal(size=(T, H)), rng.normal(size=H), rng.normal(size=(T, H))

    def loss(s, w):
        return (dy * s / np.sqrt((s ** 2).mean(-1, keepdims=True) + EPS) * w).sum()
    rstd = 1 / np.sqrt((s ** 2).mean(-1) + EPS)

    def t(a):
        return torch.tensor(a)   # helpers' to_f64 goes through fp32: compare at fp32 precision
    dx, dw, _, _ = bwd_reference(t(dy), t(s), t(w), t(rstd), None)
    h = 1e-5
    for i in range(T):
        for j in range(0, H, 5):
            d = np.zeros((T, H))
            d[i, j] = h
            assert abs((loss(s + d, w) - loss(s - d, w)) / (2 * h) - dx[i, j]) < 1e-5
    for j in range(0, H, 5):
        d = np.zeros(H)
        d[j] = h
        assert abs((loss(s, w + d) - loss(s, w - d)) / (2 * h) - dw[j]) < 1e-5


def test_refusals():
    x, r, w = inputs(4, 64)
    with pytest.raises(TypeError):
        moe_add_rmsnorm(x.float(), w)
    with pytest.raises(ValueError):
        moe_add_rmsnorm(x, w[:32])
    with pytest.raises(ValueError):
        moe_add_rmsnorm(x.t(), w)                                   # not contiguous
    with pytest.raises(ValueError):
        moe_add_rmsnorm(x, w, residual=r[:3])
    with pytest.raises(MoeError):
        moe_add_rmsnorm(x, w, eps=-1.0)
    with pytest.raises(ValueError):
        moe_add_rmsnorm(x[:, :40].contiguous(), w[:40].contiguous(), mxfp8=True)
    big = torch.empty(4 * 64 + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(MoeError):
        moe_add_rmsnorm(big[1:257].view(4, 64), w)                  # off a 16-byte boundary
    o = moe_add_rmsnorm(x, w, residual=r)
    with pytest.raises(ValueError):
        moe_add_rmsnorm_bwd(x, o.sum, w, o.rstd[:2])


def test_other_stream():
    T, H = 128, 4096
    x, r, w = inputs(T, H, seed=1)
    want = moe_add_rmsnorm(x, w, EPS, residual=r)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = moe_add_rmsnorm(x, w, EPS, residual=r)
    s.synchronize()
    assert torch.equal(got.y, want.y)


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows are read and written where they belong."""
    T, H = 530000, 4096
    assert T * H > 2 ** 31
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    rows = [0, 1, T // 2, T - 2, T - 1]
    few, r, w = inputs(len(rows), H, seed=12)
    x[rows] = few
    o = moe_add_rmsnorm(x, w, EPS, mxfp8=True)
    want = moe_add_rmsnorm(few, w, EPS, mxfp8=True)
    for n in ("y", "y_q", "y_sf", "rstd"):
        assert torch.equal(getattr(o, n)[rows], getattr(want, n)), n
    assert (o.y[2:T // 2] == 0).all()
    dx, dw = moe_add_rmsnorm_bwd(o.y, x, w, o.rstd)
    want_dx, want_dw = moe_add_rmsnorm_bwd(want.y, few, w, want.rstd)
    assert torch.equal(dx[rows], want_dx)
    torch.testing.assert_close(dw, want_dw, rtol=1e-5, atol=1e-5)   # (the zero rows add nothing; another order)


# ------------------------------------------------------------------ quantised rows to the experts

@pytest.mark.parametrize("T,H,E,k", [(1, 128, 4, 1), (1, 7168, 256, 8), (100, 2048, 64, 6), (257, 384, 8, 2),
                                     (3000, 256, 5, 3), (70, 128, 40, 32), (5000, 512, 128, 8),
                                     (64, 3200, 1024, 32), (1000, 9216, 3, 2), (16, 128, 1, 1),
                                     (8192, 128, 256, 8), (2100, 640, 1024, 8), (4200, 256, 1024, 8)])
def test_permute_rows_equals_quantising_permute(T, H, E, k):
    """Rows quantised first and permuted after = quantised by the permutation, bit for bit."""
    rows, _, _ = inputs(T, H, seed=T + E, residual=False)
    q, sf, _ = moe_grouped_quantize_mxfp8(rows)
    idx, _ = moe_route_topk(torch.randn(T, E, generator=gen(T), device="cuda"), k)
    if T > 3:
        idx[1, 0] = -1                                              # a dropped route
    ws = Workspace(T, E, k)
    want, got = PermutationMX.empty(T, H, E, k), PermutationMX.empty(T, H, E, k)
    for p in (want, got):
        for t in (p.x_q, p.src_of_row):
            t.zero_()
    moe_permute_mxfp8(rows, idx, E, ws, out=want)
    moe_permute_rows_mxfp8(q, sf, idx, E, ws, out=got)
    for n in ("dst_of_route", "src_of_row", "group_sizes", "group_offsets"):
        assert torch.equal(getattr(got, n), getattr(want, n)), n
    assert torch.equal(got.x_q, want.x_q)
    assert torch.equal(got.x_sf, want.x_sf)
    assert ws.read_error() == 0


def test_permute_rows_bad_id_and_empty():
    T, H, E, k = 6, 128, 4, 2
    q = torch.zeros(T, H, dtype=torch.uint8, device="cuda")
    sf = torch.zeros(T, H // 32, dtype=torch.uint8, device="cuda")
    idx = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    ws = Workspace(T, E, k)
    p = moe_permute_rows_mxfp8(q, sf, idx, E, ws)
    assert int(p.group_offsets[-1]) == 0 and (p.dst_of_route == -1).all() and ws.read_error() == 0
    idx[2, 1] = 9
    p = moe_permute_rows_mxfp8(q, sf, idx, E, ws)
    assert ws.read_error() == 1
    ws0 = Workspace(0, E, k)
    p = moe_permute_rows_mxfp8(q[:0], sf[:0], idx[:0], E, ws0)
    assert (p.group_sizes == 0).all()
    with pytest.raises(ValueError):
        moe_permute_rows_mxfp8(q, sf[:, :2].contiguous(), idx, E, ws)
    with pytest.raises(ValueError):
        moe_permute_rows_mxfp8(q, sf, idx, E, ws, out=PermutationMX.empty(T - 1, H, E, k))   # too small


def test_forward_mx_takes_quantised_rows():
    """MoeForwardMX on (codes, scales) = on the bf16 rows that they were quantised from."""
    T, H, F, E, k = 200, 256, 384, 8, 2
    g = gen(4)
    rows, _, _ = inputs(T, H, seed=4, residual=False)
    q, sf, _ = moe_grouped_quantize_mxfp8(rows)
    W = [torch.randn(E, a, b, generator=g, device="cuda", dtype=torch.bfloat16) * 0.02
         for a, b in ((H, F), (H, F), (F, H))]
    mw = MxWeights(*W)
    lg = torch.randn(T, E, generator=g, device="cuda")
    m = MoeForwardMX(T, H, F, E, k)
    a = m((q, sf), lg, mw).clone()
    b = m(rows, lg, mw)
    assert torch.equal(a, b)

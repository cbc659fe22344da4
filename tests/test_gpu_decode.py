"""moe_decode / moe_decode_mxfp8 (the whole layer for a few tokens) against the definition in 64 bits.

Bounds.  The output's bf16 rounding (half a step) aside, the layer keeps fp32 or better up to
the end on bf16 weights: fp32 accumulation over at most H or F terms and the fast exponential
stay below 1e-4 of the terms' size, far inside TOL = 2e-3 * RMS.  On MXFP8 weights x enters
exactly to about 2^-8 of a block's smallest normals and h as two E4M3 terms (relative rms error
0.026^2 = 7e-4 an element, averaged over the sum): five times that is 3.4e-3, inside
TOL_MX = 6e-3 * RMS."""
import numpy as np
import pytest
import torch

from helpers import assert_close_rms
from mixture_experts_ffn_warp_gb300 import (DecodeWorkspace, MoeDecode, MoeDecodeMX, MoeForward, MxWeights, moe_decode,
                                            moe_dequantize_weights_mxfp8, moe_route_topk, moe_route_topk_sigmoid)
from mixture_experts_ffn_warp_gb300._binding import DEVERR_TIMEOUT, MoeError

pytestmark = pytest.mark.gpu
TOL, TOL_MX = 2e-3, 6e-3


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def make(T, H, F, E, seed=0, wscale=0.05):
    g = gen(seed)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    lg = torch.randn(T, E, generator=g, device="cuda")
    W = [(torch.randn(E, a, b, generator=g, device="cuda") * wscale).to(torch.bfloat16)
         for a, b in ((H, F), (H, F), (F, H))]
    return x, lg, W


def reference(x, W, idx, w, clamp=None):
    x, idx, w = x.double(), idx.long(), w.double()
    out = torch.zeros(x.shape[0], W[2].shape[2], dtype=torch.float64, device=x.device)
    for e in idx.unique().tolist():
        t, j = torch.nonzero(idx == e, as_tuple=True)
        g, u = x[t] @ W[0][e].double(), x[t] @ W[1][e].double()
        if clamp is not None:
            g, u = g.clamp(clamp[0], clamp[1]), u.clamp(clamp[2], clamp[3])
        y = (g * torch.sigmoid(g) * u) @ W[2][e].double()
        out.index_add_(0, t, w[t, j].unsqueeze(1) * y)
    return out.cpu().numpy()


def check(out, ref, mx=False, what=""):
    assert_close_rms(out.double().cpu().numpy(), ref, TOL_MX if mx else TOL, what, bf16_out=True)


SHAPES = [  # T, H, F, E, k
    (1, 128, 128, 1, 1), (1, 128, 256, 8, 2), (1, 512, 384, 8, 8), (2, 256, 128, 4, 1), (7, 384, 640, 16, 3),
    (15, 256, 256, 3, 2), (16, 256, 256, 8, 2), (17, 256, 256, 8, 2), (31, 640, 384, 5, 5), (32, 128, 512, 64, 4),
    (33, 1152, 128, 8, 2), (48, 256, 896, 10, 7), (49, 256, 128, 2, 1), (63, 512, 256, 32, 6), (64, 384, 384, 4, 4),
    (64, 256, 256, 1, 1), (64, 128, 128, 300, 8), (3, 128, 128, 1024, 32), (64, 128, 128, 64, 32),
    (1, 2048, 1408, 64, 6), (13, 2048, 1408, 64, 6), (5, 4096, 2048, 16, 8), (64, 2048, 1408, 16, 6),
]


@pytest.mark.parametrize("T,H,F,E,k", SHAPES)
@pytest.mark.parametrize("mx", [False, True])
def test_shapes(T, H, F, E, k, mx):
    x, lg, W = make(T, H, F, E, seed=T + E)
    if mx:
        mw = MxWeights(*W)
        W = mw.dequantized()
        m = MoeDecodeMX(T, H, F, E, k)
        out = m(x, lg, mw)
    else:
        m = MoeDecode(T, H, F, E, k)
        out = m(x, lg, *W)
    assert m.ws.read_error() == 0
    idx, w = moe_route_topk(lg, k)
    assert torch.equal(m.topk_idx, idx)
    torch.testing.assert_close(m.topk_w, w, rtol=1e-6, atol=0)
    check(out, reference(x, W, idx, w), mx)
    # again on the same workspace: the same bits
    first = out.clone()
    again = m(x, lg, mw) if mx else m(x, lg, *W)
    assert torch.equal(again, first) and m.ws.read_error() == 0


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("bias", [True, False])
def test_sigmoid_router(mx, normalize, bias):
    T, H, F, E, k = 11, 256, 384, 40, 5
    x, lg, W = make(T, H, F, E, seed=2)
    b = torch.randn(E, generator=gen(9), device="cuda") * 0.3 if bias else None
    kw = dict(router="sigmoid", expert_bias=b, normalize=normalize)
    idx, w = moe_route_topk_sigmoid(lg, k, b, normalize)
    if mx:
        mw = MxWeights(*W)
        m = MoeDecodeMX(T, H, F, E, k, **kw)
        out = m(x, lg, mw)
        W = mw.dequantized()
    else:
        m = MoeDecode(T, H, F, E, k, **kw)
        out = m(x, lg, *W)
    assert torch.equal(m.topk_idx, idx)
    torch.testing.assert_close(m.topk_w, w, rtol=1e-6, atol=0)
    check(out, reference(x, W, idx, w), mx)


@pytest.mark.parametrize("mx", [False, True])
def test_masked_logits_and_ties(mx):
    """Rows whose logits leave no expert (all -inf: weights 0, output 0), one expert, ties (the
    lowest id), NaN (ranked last), signed zeros."""
    T, H, F, E, k = 9, 256, 256, 12, 3
    x, lg, W = make(T, H, F, E, seed=3)
    lg[0] = float("-inf")
    lg[1] = float("-inf")
    lg[1, 7] = 0.3                                  # one expert: the others rank after it with weight 0
    lg[2] = 1.5                                     # all equal
    lg[3] = 0.0
    lg[3, ::2] = -0.0
    lg[4, :6] = float("nan")
    lg[5] = torch.finfo(torch.float32).min
    lg[6, 3] = 80.0                                 # the others' weights underflow
    mw = MxWeights(*W) if mx else None
    m = (MoeDecodeMX if mx else MoeDecode)(T, H, F, E, k)
    out = m(x, lg, mw) if mx else m(x, lg, *W)
    idx, w = moe_route_topk(lg, k)
    assert torch.equal(m.topk_idx, idx)
    torch.testing.assert_close(m.topk_w, w, rtol=1e-6, atol=0)
    assert (out[0] == 0).all()
    assert idx[1, 0] == 7 and float(w[1, 0]) == 1.0 and idx[2].tolist() == [0, 1, 2] and idx[3].tolist() == [0, 1, 2]
    check(out, reference(x, mw.dequantized() if mx else W, idx, w), mx)


@pytest.mark.parametrize("mx", [False, True])
def test_infinities_stay_where_they_belong(mx):
    """A token with an infinity or a NaN leaves the others alone; so does an expert whose weights
    hold one, for the tokens that did not choose it (bf16 weights: MXFP8 codes of the quantiser
    are finite)."""
    T, H, F, E, k = 20, 256, 256, 6, 2
    x, lg, W = make(T, H, F, E, seed=4)
    bad_expert = 2
    if not mx:
        W[0][bad_expert, 5, 9] = float("nan")
        W[2][bad_expert, 100, 7] = float("inf")
    x[4, 17] = float("nan")
    x[11, 200] = float("inf")
    mw = MxWeights(*W) if mx else None
    m = (MoeDecodeMX if mx else MoeDecode)(T, H, F, E, k)
    out = m(x, lg, mw) if mx else m(x, lg, *W)
    idx, w = moe_route_topk(lg, k)
    assert torch.equal(m.topk_idx, idx)
    tokens = [t for t in range(T) if t not in (4, 11) and (mx or bad_expert not in idx[t].tolist())]
    assert 5 < len(tokens) < T
    ref = reference(x[tokens], mw.dequantized() if mx else W, idx[tokens], w[tokens])
    check(out[tokens], ref, mx)
    assert not torch.isfinite(out[4]).any()
    assert m.ws.read_error() == 0


@pytest.mark.parametrize("mx", [False, True])
def test_clamp(mx):
    T, H, F, E, k = 6, 256, 384, 8, 2
    x, lg, W = make(T, H, F, E, seed=5, wscale=0.3)
    clamp = (float("-inf"), 1.5, -1.0, 1.25)
    mw = MxWeights(*W) if mx else None
    m = (MoeDecodeMX if mx else MoeDecode)(T, H, F, E, k, swiglu_clamp=clamp)
    out = m(x, lg, mw) if mx else m(x, lg, *W)
    idx, w = moe_route_topk(lg, k)
    ref = reference(x, mw.dequantized() if mx else W, idx, w, clamp)
    check(out, ref, mx)
    free = reference(x, mw.dequantized() if mx else W, idx, w)
    assert np.abs(free - ref).max() > 0.1 * np.sqrt((ref ** 2).mean())


@pytest.mark.parametrize("mx", [False, True])
def test_fewer_tokens_than_the_layer_holds(mx):
    """One layer, calls of changing size in a row: nothing of a call is left for the next."""
    H, F, E, k = 512, 384, 24, 4
    m = (MoeDecodeMX if mx else MoeDecode)(64, H, F, E, k)
    _, _, W = make(1, H, F, E, seed=6)
    mw = MxWeights(*W) if mx else None
    Wr = mw.dequantized() if mx else W
    for i, T in enumerate((64, 1, 40, 16, 2, 64, 0, 17)):
        x, lg, _ = make(T, H, 128, E, seed=20 + i)
        out = m(x, lg, mw) if mx else m(x, lg, *W)
        assert out.shape == (T, H)
        if T:
            idx, w = moe_route_topk(lg, k)
            assert torch.equal(m.topk_idx, idx)
            check(out, reference(x, Wr, idx, w), mx, f"T={T}")
    assert m.ws.read_error() == 0
    with pytest.raises(ValueError):
        x, lg, _ = make(65, H, 128, E)
        m(x, lg, mw) if mx else m(x, lg, *W)


def test_agrees_with_the_large_batch_layer():
    T, H, F, E, k = 24, 1024, 512, 16, 4
    x, lg, W = make(T, H, F, E, seed=7)
    a = MoeDecode(T, H, F, E, k)(x, lg, *W)
    b = MoeForward(T, H, F, E, k)(x, lg, *W)
    # MoeForward rounds h and y to bf16: its own bar against the exact layer
    assert_close_rms(a.double().cpu().numpy(), b.double().cpu().numpy(), 2e-2, bf16_out=True)


def test_graph_and_streams():
    """Captured and replayed on new values; two layers with their own workspaces on two streams at once."""
    T, H, F, E, k = 3, 512, 512, 8, 2
    x, lg, W = make(T, H, F, E, seed=8)
    m = MoeDecode(T, H, F, E, k)
    m(x, lg, *W)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = m(x, lg, *W)
    x2, lg2, _ = make(T, H, 128, E, seed=9)
    x.copy_(x2)
    lg.copy_(lg2)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    idx, w = moe_route_topk(lg, k)
    want = reference(x, W, idx, w)
    check(out, want)
    m2 = MoeDecode(T, H, F, E, k)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(s1):
            o1 = m(x, lg, *W)
        with torch.cuda.stream(s2):
            o2 = m2(x, lg, *W)
    torch.cuda.synchronize()
    check(o1, want)
    assert torch.equal(o1, o2)
    assert m.ws.read_error() == 0 and m2.ws.read_error() == 0


def test_refusals():
    T, H, F, E, k = 2, 128, 256, 4, 2
    x, lg, W = make(T, H, F, E)
    ws = DecodeWorkspace(T, H, F, E, k)
    with pytest.raises(TypeError):
        moe_decode(x.float(), lg, *W, k, ws)
    with pytest.raises(TypeError):
        moe_decode(x, lg.double(), *W, k, ws)
    with pytest.raises(ValueError):
        moe_decode(x, lg[:, :3].contiguous(), *W, k, ws)
    with pytest.raises(ValueError):
        moe_decode(x, lg, W[0], W[1], W[2].transpose(1, 2), k, ws)
    with pytest.raises(MoeError):
        moe_decode(x, lg, *W, 5, ws)                     # k > E
    big = make(40, H, F, E)
    with pytest.raises(MoeError):
        moe_decode(big[0], big[1], *W, k, ws)            # a workspace for 2 tokens
    with pytest.raises(ValueError):
        DecodeWorkspace(65, H, F, E, k)
    with pytest.raises(ValueError):
        MoeDecode(T, H, F, E, k, router="hash")


@pytest.mark.parametrize("T", [4, 40])
@pytest.mark.parametrize("mx", [False, True])
def test_wait_timeout_then_recovery(mx, T):
    """With the device waits limited to 1 ns the call reports the timeout instead of finishing; after the
    workspace is initialised again the same call is right (no trap, no hang, nothing left allocated)."""
    H, F, E, k = 512, 512, 8, 2
    x, lg, W = make(T, H, F, E, seed=10)
    mw = MxWeights(*W) if mx else None
    m = (MoeDecodeMX if mx else MoeDecode)(T, H, F, E, k)
    m.ws.set_wait_limit(1)
    m(x, lg, mw) if mx else m(x, lg, *W)
    torch.cuda.synchronize()
    assert m.ws.read_error() & DEVERR_TIMEOUT
    m.ws.reset()
    out = m(x, lg, mw) if mx else m(x, lg, *W)
    assert m.ws.read_error() == 0
    idx, w = moe_route_topk(lg, k)
    check(out, reference(x, mw.dequantized() if mx else W, idx, w), mx)


def test_offsets_past_32_bits():
    """Expert weights of more than 2^31 elements a matrix: the last experts are read right."""
    T, H, F, E, k = 3, 7168, 2048, 256, 4
    assert E * H * F > 2 ** 31
    g = gen(11)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    lg = torch.randn(T, E, generator=g, device="cuda")
    lg[:, -6:] += 20.0
    W = [torch.empty(E, a, b, dtype=torch.bfloat16, device="cuda") for a, b in ((H, F), (H, F), (F, H))]
    for w in W:
        for e in range(E):
            w[e] = torch.randn(w.shape[1:], generator=g, device="cuda", dtype=torch.bfloat16) * 0.02
    idx, w = moe_route_topk(lg, k)
    assert int(idx.min()) >= E - 6
    out = MoeDecode(T, H, F, E, k)(x, lg, *W)
    check(out, reference(x, W, idx, w))
    mw = MxWeights(*W)
    for i, (q, sf, K, N) in enumerate(((mw.Wg_q, mw.Wg_sf, H, F), (mw.Wu_q, mw.Wu_sf, H, F), (mw.Wd_q, mw.Wd_sf, F, H))):
        n = K * N
        for e in idx.unique().tolist():             # the values of the hit experts' codes
            W[i][e] = moe_dequantize_weights_mxfp8(q[e * n:(e + 1) * n], sf[e * n // 32:(e + 1) * n // 32], 1, K, N)[0]
    out = MoeDecodeMX(T, H, F, E, k)(x, lg, mw)
    check(out, reference(x, W, idx, w), mx=True)

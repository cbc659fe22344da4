"""Operators around a mixture-of-experts FFN block: the cases they are timed on, and their plain forms.

Five operators:

  decode        a whole MoE layer for a few tokens (1 to 64), bf16 expert weights: top-k routing of
                fp32 logits, gate / up products, SwiGLU, down product, weighted sum over the experts
  decode_mx     the same layer on expert weights kept in MXFP8 (E4M3 codes, one UE8M0 scale per 32
                elements of the contraction), activations in bf16
  norm          s = x + residual, y = s * rsqrt(mean(s^2) + eps) * weight; s in bf16, y in bf16 and / or
                MXFP8 along the row
  norm_bwd      its gradient: dx (of x and of the residual alike) and the weight's
  permute_rows  rows that are already MXFP8 moved to expert-contiguous order, their scales into the
                block-scaled product's operand layout

`own` selects who computes: False, elementary torch operations in 32 bits (this file alone); True, the
framework's kernels."""
import math

import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # one token through a small layer: nothing but latency (a test model, a draft model's block)
        dict(name="decode tiny 1", op="decode", T=1, H=128, F=256, E=8, k=2, router="softmax"),
        # one sequence being generated, few large experts: two experts' weights read once
        dict(name="decode mixtral 1", op="decode", T=1, H=4096, F=14336, E=8, k=2, router="softmax"),
        # a small odd batch on fine-grained experts with the sigmoid router: most experts hit, one or two tokens each
        dict(name="decode fine_grained 13", op="decode", T=13, H=2048, F=1408, E=64, k=6, router="sigmoid"),
        # a serving batch on many experts: nearly all of them read
        dict(name="decode skewed 64", op="decode", T=64, H=4096, F=2048, E=128, k=8, router="softmax"),
        # one sequence on 8-bit weights of a large sparse layer: 8 experts of 256
        dict(name="decode_mx dsv3 1", op="decode_mx", T=1, H=7168, F=2048, E=256, k=8, router="sigmoid"),
        # an odd batch on 8-bit fine-grained experts
        dict(name="decode_mx fine_grained 37", op="decode_mx", T=37, H=2048, F=1408, E=64, k=6, router="softmax"),
        # the norm before the layer: one generated token
        dict(name="norm 1", op="norm", T=1, H=4096, bf16=True, mx=False, residual=True),
        # a prompt's tokens, for the 8-bit layer and its router: both outputs
        dict(name="norm dsv3 8192 mx", op="norm", T=8192, H=7168, bf16=True, mx=True, residual=True),
        # a short odd training batch
        dict(name="norm_bwd 333", op="norm_bwd", T=333, H=2048, residual=True),
        # the training step's batch
        dict(name="norm_bwd mixtral 8192", op="norm_bwd", T=8192, H=4096, residual=True),
        # a short prompt's quantised rows to the experts
        dict(name="permute_rows 100", op="permute_rows", T=100, H=2048, E=64, k=6),
        # a long prompt's
        dict(name="permute_rows dsv3 8192", op="permute_rows", T=8192, H=7168, E=256, k=8),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, unit, lo, hi):
    """unit * [lo, hi]; the one width that this repository's layers do not come in moves up a step."""
    n = unit * _log_int(rng, lo, hi)
    return n + unit if n == 24 * 128 else n


def draw(rng):
    op = rng.choice(["decode", "decode", "decode_mx", "decode_mx", "norm", "norm_bwd", "permute_rows"])
    if op in ("decode", "decode_mx"):
        T = _log_int(rng, 1, 64)
        H, F = _width(rng, 128, 1, 56), _width(rng, 128, 1, 112)
        E = _log_int(rng, 2, 256)
        while 3 * E * H * F > 3_200_000_000:   # the largest listed layer's weights
            E //= 2
        k = rng.randint(1, min(8, E))
        return dict(op=op, T=T, H=H, F=F, E=E, k=k, router=rng.choice(["softmax", "sigmoid"]))
    if op == "permute_rows":
        E = _log_int(rng, 4, 256)
        return dict(op=op, T=_log_int(rng, 1, 8192), H=_width(rng, 128, 1, 56), E=E, k=rng.randint(1, min(8, E)))
    T = _log_int(rng, 1, 8192)
    if op == "norm":
        mx = rng.random() < 0.5
        H = _width(rng, 32, 4, 224) if mx else _width(rng, 8, 16, 896)
        return dict(op=op, T=T, H=H, bf16=not mx or rng.random() < 0.5, mx=mx, residual=rng.random() < 0.75)
    return dict(op=op, T=T, H=_width(rng, 8, 16, 896), residual=rng.random() < 0.75)


def work(case):
    c, T, H = case, case["T"], case["H"]
    if c["op"] in ("decode", "decode_mx"):
        F, E, k = c["F"], c["E"], c["k"]
        hit = E * (1.0 - (1.0 - k / E) ** T)             # distinct experts that T tokens' top-k reach, on average
        per = 3.0 * H * F * (2.0 if c["op"] == "decode" else 1.0 + 1.0 / 32.0)
        return {"bytes": hit * per + T * (4.0 * H + 4.0 * E + 8.0 * k), "flops": 6.0 * T * k * H * F}
    if c["op"] == "norm":
        per = 2.0 + (4.0 if c["residual"] else 0.0) + (2.0 if c["bf16"] else 0.0) + (33.0 / 32.0 if c["mx"] else 0.0)
        return {"bytes": T * (H * per + 4.0) + 2.0 * H, "flops": 8.0 * T * H}
    if c["op"] == "norm_bwd":
        return {"bytes": T * (H * (6.0 + (2.0 if c["residual"] else 0.0)) + 4.0) + 6.0 * H, "flops": 12.0 * T * H}
    k = c["k"]
    row = H * 33.0 / 32.0
    return {"bytes": T * row * (1.0 + k) + T * k * 12.0, "flops": 0.0}


# ------------------------------------------------------------------------------------ inputs

def _mx_quantise(v):
    """MXFP8 along the last dimension, blocks of 32: (E4M3 codes, UE8M0 scale bytes), both uint8. The scale is
    the smallest 2^X with the block's largest magnitude at most 448 * 2^X."""
    b = v.reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
    m, e = torch.frexp(b.abs().amax(-1))                 # amax = m * 2^e, m in [0.5, 1)
    X = e - 9 + (m > 0.875).to(e.dtype)
    X = torch.where(m == 0, torch.full_like(X, -127), X).clamp(-127, 127)
    scaled = torch.ldexp(b, -X.unsqueeze(-1)).clamp(-448.0, 448.0)
    codes = scaled.to(torch.float8_e4m3fn).view(torch.uint8).reshape(v.shape)
    return codes, (X + 127).to(torch.uint8)


def _mx_values(codes, scales, dtype=torch.float32):
    v = codes.view(torch.float8_e4m3fn).to(dtype)
    s = torch.exp2(scales.to(dtype) - 127.0)
    return (v.reshape(*scales.shape, 32) * s.unsqueeze(-1)).reshape(codes.shape)


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _draw_decode(case, g):
    """x after a norm, the router's logits and its selection bias."""
    T, H, E = case["T"], case["H"], case["E"]
    return {"x": torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16),
            "logits": torch.randn(T, E, generator=g, device="cuda"),
            "bias": torch.randn(E, generator=g, device="cuda") * 0.05 if case["router"] == "sigmoid" else None}


def _draw_weights(case, g):
    H, F = case["H"], case["F"]
    for e in range(case["E"]):
        yield e, [torch.randn(a, b, generator=g, device="cuda", dtype=torch.bfloat16) * 0.02
                  for a, b in ((H, F), (H, F), (F, H))]


# The expert weights are drawn one expert at a time, in one order for every form.
def _weights_bf16(case, g):
    H, F, E = case["H"], case["F"], case["E"]
    w = [torch.empty(E, a, b, dtype=torch.bfloat16, device="cuda") for a, b in ((H, F), (H, F), (F, H))]
    for e, ws in _draw_weights(case, g):
        for dst, src in zip(w, ws):
            dst[e] = src
    return w


def _weights_mx(case, g):
    """Codes and scales of each matrix with the contraction last: gate, up [E, F, H], down [E, H, F]."""
    H, F, E = case["H"], case["F"], case["E"]
    w = [(torch.empty(E, n, c, dtype=torch.uint8, device="cuda"),
          torch.empty(E, n, c // 32, dtype=torch.uint8, device="cuda")) for c, n in ((H, F), (H, F), (F, H))]
    for e, ws in _draw_weights(case, g):
        for (codes, scales), src in zip(w, ws):
            codes[e], scales[e] = _mx_quantise(src.t().float())
    return w


def _draw_norm(case, g):
    """A layer's output and the residual stream, some of whose channels are much larger than the rest."""
    T, H = case["T"], case["H"]
    big = 1.0 + 20.0 * (torch.rand(H, generator=g, device="cuda") < 0.01).float()
    s = {"x": torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16),
         "weight": (1.0 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)}
    r = 2.0 * torch.randn(T, H, generator=g, device="cuda") * big
    s["residual"] = r.to(torch.bfloat16) if case["residual"] else None
    if case["op"] == "norm_bwd":
        s["dy"] = s.pop("x")
        s["sum"] = r.to(torch.bfloat16)
        s["d_sum"] = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16) if case["residual"] else None
        s["rstd"] = torch.rsqrt(s["sum"].float().square().mean(-1) + EPS)
        s.pop("residual")
    return s


def _draw_rows(case, g):
    T, H, E, k = case["T"], case["H"], case["E"], case["k"]
    codes, scales = _mx_quantise(torch.randn(T, H, generator=g, device="cuda"))
    idx = torch.rand(T, E, generator=g, device="cuda").argsort(-1)[:, :k].to(torch.int32).contiguous()
    return {"x_q": codes, "x_sf": scales, "idx": idx}


def prepare(case, seed):
    g, op = _generator(seed), case["op"]
    if op in ("decode", "decode_mx"):
        s = _draw_decode(case, g)
        T, H, F, E, k = (case[n] for n in "THFEk")
        if own:
            import mixture_experts_ffn_warp_gb300 as moe
            w = _weights_bf16(case, g)
            kind = moe.MoeDecode if op == "decode" else moe.MoeDecodeMX
            s["layer"] = kind(T, H, F, E, k, router=case["router"], expert_bias=s["bias"])
            s["weights"] = w if op == "decode" else [moe.MxWeights(*w)]
        else:
            s["weights"] = _weights_bf16(case, g) if op == "decode" else _weights_mx(case, g)
    elif op == "permute_rows":
        s = _draw_rows(case, g)
        if own:
            import mixture_experts_ffn_warp_gb300 as moe
            T, H, E, k = (case[n] for n in "THEk")
            s["ws"] = moe.Workspace(T, E, k)
            s["out"] = moe.PermutationMX.empty(T, H, E, k)
    else:
        s = _draw_norm(case, g)
        if own:
            import mixture_experts_ffn_warp_gb300 as moe
            T, H = case["T"], case["H"]
            if op == "norm":
                s["out"] = moe.NormOutput.empty(T, H, bf16=case["bf16"], mxfp8=case["mx"], residual=case["residual"])
            else:
                s["ws"] = moe.NormWorkspace(T, H)
                s["dx"] = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
                s["dweight"] = torch.empty(H, dtype=torch.float32, device="cuda")
    s["case"] = dict(case)
    return s


# ------------------------------------------------------------------------------------ plain forms

def _plain_route(s, c):
    k = c["k"]
    if c["router"] == "softmax":
        idx = s["logits"].sort(dim=-1, descending=True, stable=True).indices[:, :k]
        v = s["logits"].gather(1, idx)
        e = torch.exp(v - v[:, :1])
        w = e / e.sum(-1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-s["logits"]))
        idx = (score + s["bias"]).sort(dim=-1, descending=True, stable=True).indices[:, :k]
        v = score.gather(1, idx)
        w = v / (v.sum(-1, keepdim=True) + 1e-20)
    return idx, w


def _plain_decode(s, c):
    idx, w = _plain_route(s, c)
    x = s["x"].float()
    if c["op"] == "decode":
        matrix = lambda i, sel: s["weights"][i][sel].float()                     # noqa: E731  [n, contraction, out]
    else:
        matrix = lambda i, sel: _mx_values(s["weights"][i][0][sel], s["weights"][i][1][sel]).transpose(-1, -2)  # noqa: E731
    T, k, E = c["T"], c["k"], c["E"]
    if T * k <= E:                                    # few routes: each route's own expert
        sel = idx.reshape(-1)
        xr = x.repeat_interleave(k, 0).unsqueeze(1)   # [T*k, 1, H]
        g, u = xr @ matrix(0, sel), xr @ matrix(1, sel)
        y = (g / (1.0 + torch.exp(-g)) * u) @ matrix(2, sel)
        out = (y.reshape(T, k, -1) * w.unsqueeze(-1)).sum(1)
    else:                                             # every expert on every token, weighted by its share (0 where not routed)
        every = slice(None)
        share = torch.zeros(T, E, device=x.device).scatter(1, idx, w)
        g, u = x @ matrix(0, every), x @ matrix(1, every)
        h = g / (1.0 + torch.exp(-g)) * u * share.t().unsqueeze(-1)
        out = (h @ matrix(2, every)).sum(0)
    return {"out": out.to(torch.bfloat16), "topk_idx": idx.to(torch.int32), "topk_w": w}


def _plain_norm(s, c):
    v = s["x"].float()
    if s["residual"] is not None:
        v = v + s["residual"].float()
    rstd = torch.rsqrt(v.square().mean(-1) + EPS)
    y = v * rstd.unsqueeze(-1) * s["weight"].float()
    r = {"rstd": rstd}
    if s["residual"] is not None:
        r["sum"] = v.to(torch.bfloat16)
    if c["bf16"]:
        r["y"] = y.to(torch.bfloat16)
    if c["mx"]:
        codes, scales = _mx_quantise(y)
        r["y_q"], r["y_sf"] = codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)
    return r


def _plain_norm_bwd(s, c):
    dy, v, rstd = s["dy"].float(), s["sum"].float(), s["rstd"].unsqueeze(-1)
    xhat = v * rstd
    wdy = dy * s["weight"].float()
    dx = rstd * (wdy - xhat * (wdy * xhat).mean(-1, keepdim=True))
    if s["d_sum"] is not None:
        dx = dx + s["d_sum"].float()
    return {"dx": dx.to(torch.bfloat16), "dweight": (dy * xhat).sum(0)}


def _plain_permute_rows(s, c):
    T, H, E, k = (c[n] for n in "THEk")
    R = T * k
    e = s["idx"].reshape(-1).long()
    src = torch.sort(e, stable=True).indices                  # route of each row: expert by expert, routes in order
    dst = torch.empty_like(src)
    dst[src] = torch.arange(R, device=e.device)
    sizes = (e.unsqueeze(0) == torch.arange(E, device=e.device).unsqueeze(1)).sum(1)
    offsets = torch.cat([torch.zeros(1, dtype=torch.long, device=e.device), sizes.cumsum(0)])
    tiles = (sizes + 127) // 128                              # 128-row tiles of each group's scales
    first = tiles.cumsum(0) - tiles
    row_e = e[src]
    i = torch.arange(R, device=e.device) - offsets[row_e]     # row inside its group
    kb = torch.arange(H // 32, device=e.device)
    atom = (first[row_e] + i // 128).unsqueeze(1) * (H // 128) + kb // 4
    at = atom * 512 + ((i % 32) * 16 + (i % 128) // 32 * 4).unsqueeze(1) + kb % 4
    sf = torch.zeros(((R + 127) // 128 + E) * (H // 128) * 512, dtype=torch.uint8, device=e.device)
    sf[at] = s["x_sf"][src // k]
    as_int = lambda v: v.to(torch.int32)                      # noqa: E731
    return {"x_q": s["x_q"][src // k], "x_sf": sf, "dst_of_route": as_int(dst).reshape(T, k), "src_of_row": as_int(src),
            "group_sizes": as_int(sizes), "group_offsets": as_int(offsets)}


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"decode": _plain_decode, "decode_mx": _plain_decode, "norm": _plain_norm, "norm_bwd": _plain_norm_bwd,
                "permute_rows": _plain_permute_rows}[op](s, c)
    import mixture_experts_ffn_warp_gb300 as moe
    if op in ("decode", "decode_mx"):
        m = s["layer"]
        out = m(s["x"], s["logits"], *s["weights"])
        return {"out": out, "topk_idx": m.topk_idx, "topk_w": m.topk_w}
    if op == "norm":
        n = moe.moe_add_rmsnorm(s["x"], s["weight"], EPS, residual=s["residual"], out=s["out"])
        r = {"rstd": n.rstd}
        if s["residual"] is not None:
            r["sum"] = n.sum
        if c["bf16"]:
            r["y"] = n.y
        if c["mx"]:
            r["y_q"], r["y_sf"] = n.y_q.view(torch.float8_e4m3fn), n.y_sf.view(torch.float8_e8m0fnu)
        return r
    if op == "norm_bwd":
        dx, dweight = moe.moe_add_rmsnorm_bwd(s["dy"], s["sum"], s["weight"], s["rstd"], d_sum=s["d_sum"], dx=s["dx"],
                                              dweight=s["dweight"], ws=s["ws"])
        return {"dx": dx, "dweight": dweight}
    p = moe.moe_permute_rows_mxfp8(s["x_q"], s["x_sf"], s["idx"], c["E"], s["ws"], out=s["out"])
    return {"x_q": p.x_q, "x_sf": p.x_sf, "dst_of_route": p.dst_of_route, "src_of_row": p.src_of_row,
            "group_sizes": p.group_sizes, "group_offsets": p.group_offsets}


# ------------------------------------------------------------------------------------ 64 bits

def _exact_decode(case, seed):
    """Token by expert, from the definition; the experts' weights are drawn again one at a time."""
    g = _generator(seed)
    s = _draw_decode(case, g)
    T, H, E, k = (case[n] for n in "THEk")
    lg = s["logits"].double()
    rank = lg if case["router"] == "softmax" else torch.sigmoid(lg) + s["bias"].double()
    idx = torch.argsort(-rank, dim=1, stable=True)[:, :k]
    if case["router"] == "softmax":
        w = torch.softmax(torch.gather(lg, 1, idx), 1)
    else:
        w = torch.gather(torch.sigmoid(lg), 1, idx)
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    x = s["x"].double()
    for e, ws in _draw_weights(case, g):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        if t.numel() == 0:
            continue
        if case["op"] == "decode_mx":
            ws = [_mx_values(*_mx_quantise(m.t().float()), dtype=torch.float64).t() for m in ws]
        wg, wu, wd = (m.double() for m in ws)
        gate, up = x[t] @ wg, x[t] @ wu
        out.index_add_(0, t, w[t, j].unsqueeze(1) * ((gate * torch.sigmoid(gate) * up) @ wd))
    return {"out": out, "topk_idx": None, "topk_w": w}


def exact(case, seed):
    op = case["op"]
    if op in ("decode", "decode_mx"):
        return _exact_decode(case, seed)
    if op == "permute_rows":
        return None                       # whole numbers and copied bytes
    s = _draw_norm(case, _generator(seed))
    if op == "norm":
        v = s["x"].double() + (s["residual"].double() if case["residual"] else 0.0)
        ms = torch.einsum("th,th->t", v, v) / case["H"]
        y = v * s["weight"].double() / torch.sqrt(ms + EPS).unsqueeze(1)
        r = {"rstd": 1.0 / torch.sqrt(ms + EPS)}
        if case["residual"]:
            r["sum"] = v
        if case["bf16"]:
            r["y"] = y
        if case["mx"]:
            codes, scales = _mx_quantise(y)
            r["y_q"], r["y_sf"] = codes.view(torch.float8_e4m3fn).double(), torch.exp2(scales.double() - 127.0)
        return r
    v, dy, gamma, rstd = s["sum"].double(), s["dy"].double(), s["weight"].double(), s["rstd"].double()
    dot = torch.einsum("th,th,h->t", dy, v, gamma)            # <dy * weight, s>
    dx = dy * gamma * rstd.unsqueeze(1) - v * (rstd.pow(3) * dot / case["H"]).unsqueeze(1)
    if case["residual"]:
        dx = dx + s["d_sum"].double()
    return {"dx": dx, "dweight": torch.einsum("th,th,t->h", dy, v, rstd)}

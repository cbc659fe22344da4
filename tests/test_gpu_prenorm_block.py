"""The pre-norm block of examples/prenorm_block.py end to end: generation, prompt and training step
against the same block in 64 bits."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
EXAMPLE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "prenorm_block.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("prenorm_block", EXAMPLE)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def exact_block(block, x, r, W, leaf=False):
    """The block in 64 bits with autograd; the routing is taken from the logits as they are."""
    s = (x.double() + r.double()).requires_grad_(leaf)
    gamma = block.norm_weight.double().requires_grad_(leaf)
    Wr = block.W_router.double().requires_grad_(leaf)
    W = [w.double().requires_grad_(leaf) for w in W]
    y = s / torch.sqrt((s * s).mean(-1, keepdim=True) + 1e-6) * gamma
    logits = y @ Wr
    top = logits.topk(block.k, -1)
    w = torch.softmax(top.values, -1)
    share = torch.zeros_like(logits).scatter(1, top.indices, w)
    out = 0
    for e in range(block.E):
        g, u = y @ W[0][e], y @ W[1][e]
        out = out + share[:, e:e + 1] * ((g * torch.sigmoid(g) * u) @ W[2][e])
    gap = logits.sort(-1, descending=True).values
    clear = (gap[:, block.k - 1] - gap[:, block.k]) > 0.03     # tokens whose selection no rounding turns
    return out, s, gamma, Wr, W, clear


def off(a, b):
    return float((a.double() - b).norm() / b.norm())


def rows(g, T, H):
    return torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)


def test_generation_and_prompt(example):
    block = example.PreNormMoE(H=512, F=384, E=8, k=2)
    g = torch.Generator(device="cuda").manual_seed(2)
    x, r = rows(g, 200, 512), rows(g, 200, 512)
    want, s, *_, clear = exact_block(block, x, r, block.W)
    want_mx, *_ = exact_block(block, x, r, block.W_mx.dequantized())
    assert int(clear.sum()) > 100
    pick = clear.nonzero().flatten()[:33]
    few, stream = block.generate(x[pick], r[pick])
    assert off(stream, s[pick]) < 2.0 ** -8
    # y enters the layer rounded to bf16 (relative rms 1.6e-3 an element); so does the output
    assert off(few, want[pick]) < 6e-3
    few_mx, _ = block.generate(x[pick], r[pick], mx=True)
    assert off(few_mx, want_mx[pick]) < 6e-3
    prompt, _ = block.prompt(x, r)
    # E4M3 rows of y and of h: relative rms 2.6e-2 an element each
    assert off(prompt[clear], want_mx[clear]) < 8e-2


def test_training_step(example):
    block = example.PreNormMoE(H=256, F=384, E=4, k=2)
    g = torch.Generator(device="cuda").manual_seed(3)
    T = 150
    x, r, d_out, d_res = rows(g, T, 256), rows(g, T, 256), rows(g, T, 256), rows(g, T, 256)
    out, s, gamma, Wr, W, clear = exact_block(block, x, r, block.W, leaf=True)
    # tokens whose selection is not clear take no part
    x, r, d_out, d_res = x[clear], r[clear], d_out[clear], d_res[clear]
    out, s, gamma, Wr, W, clear = exact_block(block, x, r, block.W, leaf=True)
    assert bool(clear.all()) and x.shape[0] > 80
    ((out * d_out.double()).sum() + (s * d_res.double()).sum()).backward()
    got, dx, grads = block.train_step(x, r, d_out, d_res)
    assert off(got, out.detach()) < 1e-2
    # bf16 intermediates (y, h, dgu, dx_perm's sum): a few roundings of 1.6e-3 each
    assert off(dx, s.grad) < 1.5e-2
    for n, want in (("norm_weight", gamma.grad), ("W_router", Wr.grad), ("W_gate", W[0].grad), ("W_up", W[1].grad),
                    ("W_down", W[2].grad)):
        assert off(grads[n], want) < 1.5e-2, n

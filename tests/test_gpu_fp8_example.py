"""The feed-forward example: outputs and gradients against the same layers in 64 bits, training and decoding.

Tolerance. Rounding to e4m3 is off by at most 2^-4 of a value, evenly spread over half a spacing: 2.6 % of the
operand in the root mean square. A sum over a rounded operand carries that over in the Frobenius norm, and independent
roundings add in squares, so a result that n rounded operands went into is off by about 2.6 % sqrt(n); three times
that is allowed. A wrong scale, axis or operand is off by the order of 1."""

import importlib.util
import os

import pytest
import torch

import async_global_shared_gb300 as ap

pytestmark = pytest.mark.gpu

ROUNDING = 3 * 0.026


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "fp8_feed_forward.py")
    spec = importlib.util.spec_from_file_location("fp8_feed_forward", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def build(ex, width, hidden, count):
    gen = torch.Generator(device="cuda").manual_seed(5)
    layers = [ex.FeedForward(width, hidden, gen) for _ in range(count)]
    for layer in layers:
        layer.norm.copy_(1 + 0.1 * torch.randn(width, generator=gen, device="cuda"))
    return layers, gen


def plain(layers, tokens, eps):
    """The stack's h + out in 64 bits, with its weights as leaves."""
    weights = [[w.double().cpu().requires_grad_() for w in (layer.norm, layer.w1.value, layer.w2.value)] for layer in layers]
    h = tokens.double().cpu()
    out = torch.zeros_like(h)
    for norm, w1, w2 in weights:
        h = h + out
        y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + eps) * norm
        out = torch.nn.functional.silu(y @ w1.T) @ w2.T
    return h + out, out, weights


def off(got, want):
    return ((got.double().cpu() - want).norm() / want.norm()).item()


# a width and a hidden size that are no multiples of the block; few and many tokens
@pytest.mark.parametrize("tokens,width,hidden", [(1, 256, 512), (50, 200, 328), (300, 512, 1000)])
def test_outputs_and_gradients(tokens, width, hidden):
    ex = example()
    layers, gen = build(ex, width, hidden, 2)
    x = torch.randn(tokens, width, generator=gen, device="cuda")
    want, want_out, weights = plain(layers, x, ex.EPS)
    direction = torch.randn(tokens, width, generator=gen, device="cuda")
    (want * direction.double().cpu()).sum().backward()

    out, h = torch.zeros_like(x, dtype=torch.bfloat16), x
    kept = []
    for layer in layers:
        out, h, k = layer.forward(out, h)
        kept.append(k)
    # the last layer's out: four operands of its own, and four of the layer before in its input
    assert off(out, want_out.detach()) < ROUNDING * 8 ** 0.5
    dh = direction.clone()
    for i in reversed(range(2)):
        dh, grads = layers[i].backward(dh.to(torch.bfloat16), dh, kept[i])
        # the eight of the pass forward, and at most eight of the pass back
        for got, leaf in zip(grads, weights[i]):
            assert off(got, leaf.grad) < ROUNDING * 16 ** 0.5
    assert ap.ap_check() == 0


def test_inference_equals_the_training_pass():
    ex = example()
    layers, gen = build(ex, 512, 1000, 2)
    x = torch.randn(70, 512, generator=gen, device="cuda")
    out, h = torch.zeros_like(x, dtype=torch.bfloat16), x
    for layer in layers:
        out, h, _ = layer.forward(out, h)
    out2, h2 = torch.zeros_like(x, dtype=torch.bfloat16), x.clone()
    for layer in layers:
        out2, h2 = layer.infer(out2, h2)
    assert torch.equal(out, out2) and torch.equal(h, h2)


def test_training_lowers_the_loss():
    ex = example()
    layers, gen = build(ex, 256, 512, 2)
    x = torch.randn(512, 256, generator=gen, device="cuda")
    target = x.roll(1, 1)
    losses = [ex.train_step(layers, x, target, 2.0).item() for _ in range(12)]
    assert all(b < a for a, b in zip(losses, losses[1:])), losses


def test_decoding_by_graph():
    ex = example()
    layers, gen = build(ex, 384, 640, 2)
    decode = ex.Decoder(layers, 384)
    for _ in range(3):
        token = torch.randn(1, 384, generator=gen, device="cuda")
        got = decode(token).clone()
        out, h = torch.zeros(1, 384, dtype=torch.bfloat16, device="cuda"), token.clone()
        for layer in layers:
            out, h = layer.infer(out, h)
        assert torch.equal(got, h + out)

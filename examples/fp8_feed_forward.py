"""A pre-norm feed-forward layer whose matrix products run in 8-bit floating point, trained and then decoded with.

    h = x + residual;  y = norm(h);  u = y W1^T;  out = silu(u) W2^T        (out and h go on to the next layer)

Every product reads e4m3 operands with a scale for each block of 128 along the axis it sums over, so a matrix that is
summed over both ways (weights, and in training activations and gradients) is held in two forms:

    forward      u     = y    . W1      y by rows (written by the norm), W1 in tiles
                 out   = act  . W2      act by rows, W2 in tiles
    backward     dact  = dout . W2^T    dout by rows, W2 transposed in tiles
                 dW2   = dout^T . act^T dout and act by columns: what the quantiser writes transposed
                 dy    = du . W1^T, dW1 = du^T . y^T the same way
                 dx, dnorm              the norm's gradient, with the residual stream's own gradient added

The weights stay in 32 bits; their 8-bit forms are made again after each step. The residual stream is held in 32 bits,
everything else between the operators in bf16. Decoding captures one token's pass through the layers in a CUDA graph.

    python examples/fp8_feed_forward.py [--tokens 8192 --width 4096 --hidden 16384 --layers 2 --steps 10]
"""

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import async_global_shared_gb300 as ap

EPS = 1e-6
E4M3 = torch.float8_e4m3fn


def blocks(n):
    return (n + 127) // 128


class Codes:
    """Room for a rows x cols matrix in e4m3, its rows on 16-byte boundaries, and the scales of its row blocks
    (tile 1) or its 128 x 128 tiles (tile 128)."""

    def __init__(self, rows, cols, tile=1):
        pitch = (cols + 15) // 16 * 16
        self.q = torch.empty(rows, pitch, dtype=torch.uint8, device="cuda").view(E4M3)[:, :cols]
        self.s = torch.empty((rows + tile - 1) // tile, blocks(cols), device="cuda")
        self.tile = tile


def product(a, b, dtype=torch.bfloat16):
    """a b^T."""
    c = torch.empty(a.q.shape[0], b.q.shape[0], dtype=dtype, device="cuda")
    ap.ap_matmul_fp8(a.q, a.s, b.q, b.s, c, b.tile)
    return c


def both_ways(x, rows=True):
    """x by row blocks (where asked for) and its transpose by row blocks."""
    r = Codes(*x.shape) if rows else None
    t = Codes(x.shape[1], x.shape[0])
    ap.ap_quantize(x, 1, r and r.q, r and r.s, t.q, t.s)
    return r, t


class Weight:
    """An out x in weight in 32 bits, with its 8-bit tiles as it stands and transposed."""

    def __init__(self, out, inner, gen):
        self.value = torch.randn(out, inner, generator=gen, device="cuda") / inner ** 0.5
        self.codes, self.turned = Codes(out, inner, 128), Codes(inner, out, 128)
        self.lay_out()

    def lay_out(self):
        ap.ap_quantize(self.value, 128, self.codes.q, self.codes.s, self.turned.q, self.turned.s)

    def step(self, grad, rate):
        self.value.sub_(grad, alpha=rate)
        self.lay_out()


class FeedForward:
    def __init__(self, width, hidden, gen):
        self.norm = torch.ones(width, device="cuda")
        self.w1 = Weight(hidden, width, gen)
        self.w2 = Weight(width, hidden, gen)
        self.workspace = None

    def infer(self, x, residual):
        """out and the residual stream after x, which takes the residual's place."""
        y = Codes(*x.shape)
        ap.ap_rms_norm(x, self.norm, EPS, q=y.q, q_scales=y.s, residual=residual, residual_out=residual)
        act = torch.nn.functional.silu(product(y, self.w1.codes))
        a = Codes(*act.shape)
        ap.ap_quantize(act, 1, a.q, a.s)
        return product(a, self.w2.codes), residual

    def forward(self, x, residual):
        """As infer, with a residual stream of its own, and what backward needs."""
        rows, width = x.shape
        h, y, rstd = torch.empty_like(residual), torch.empty_like(x), torch.empty(rows, device="cuda")
        y8 = Codes(rows, width)
        ap.ap_rms_norm(x, self.norm, EPS, y=y, q=y8.q, q_scales=y8.s, residual=residual, residual_out=h, rstd=rstd)
        _, yt = both_ways(y, rows=False)
        u = product(y8, self.w1.codes)
        a8, at = both_ways(torch.nn.functional.silu(u))
        return product(a8, self.w2.codes), h, (h, rstd, yt, u, at)

    def backward(self, dout, dh, kept):
        """Gradient of x and residual (one and the same), in place of dh, and of the norm's weight, W1 and W2."""
        h, rstd, yt, u, at = kept
        d8, dt = both_ways(dout)
        dw2 = product(dt, at, torch.float32)
        du = torch.ops.aten.silu_backward(product(d8, self.w2.turned), u)
        d8, dt = both_ways(du)
        dw1 = product(dt, yt, torch.float32)
        dy = product(d8, self.w1.turned)
        if self.workspace is None or self.workspace.nbytes < ap.ap_rms_norm_backward_workspace(*h.shape):
            self.workspace = torch.empty(ap.ap_rms_norm_backward_workspace(*h.shape), dtype=torch.uint8, device="cuda")
        dnorm = torch.empty_like(self.norm)
        ap.ap_rms_norm_backward(dy, h, self.norm, rstd, dh, dnorm, self.workspace, dresidual=dh)
        return dh, (dnorm, dw1, dw2)


def train_step(layers, tokens, target, rate):
    """One pass forward and back over tokens (float32), towards target, and a step of every weight; the loss before it."""
    out, h = torch.zeros_like(tokens, dtype=torch.bfloat16), tokens
    kept = []
    for layer in layers:
        out, h, k = layer.forward(out, h)
        kept.append(k)
    error = h + out - target
    dh = error * (2 / error.numel())
    for layer, k in zip(reversed(layers), reversed(kept)):
        dh, (dnorm, dw1, dw2) = layer.backward(dh.to(torch.bfloat16), dh, k)
        layer.norm.sub_(dnorm, alpha=rate)
        layer.w1.step(dw1, rate)
        layer.w2.step(dw2, rate)
    return error.square().mean()


class Decoder:
    """One token's pass through the layers as a CUDA graph."""

    def __init__(self, layers, width):
        self.token = torch.zeros(1, width, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):  # attributes are set outside the capture
            self._pass(layers)
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.result = self._pass(layers)

    def _pass(self, layers):
        out, h = torch.zeros_like(self.token, dtype=torch.bfloat16), self.token.clone()
        for layer in layers:
            out, h = layer.infer(out, h)
        return h + out

    def __call__(self, token):
        self.token.copy_(token)
        self.graph.replay()
        return self.result


def timed(call, runs):
    """Milliseconds a run, after one that is not counted."""
    call()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(runs):
        result = call()
    end.record()
    end.synchronize()
    return start.elapsed_time(end) / runs, result


def main():
    args = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 8192), ("width", 4096), ("hidden", 16384), ("layers", 2), ("steps", 10)):
        args.add_argument(f"--{name}", type=int, default=value)
    a = args.parse_args()
    gen = torch.Generator(device="cuda").manual_seed(1)
    layers = [FeedForward(a.width, a.hidden, gen) for _ in range(a.layers)]
    tokens = torch.randn(a.tokens, a.width, generator=gen, device="cuda")
    target = tokens.roll(1, 1)
    rate = 1.0
    first = train_step(layers, tokens, target, rate).item()
    ms, loss = timed(lambda: train_step(layers, tokens, target, rate), a.steps)
    products = 6 * 2 * a.tokens * a.width * a.hidden * a.layers
    print(f"training: loss {first:.4f} -> {loss.item():.4f}, {ms:.2f} ms a step, {products / ms * 1e-9:.0f} TFLOP/s over all")
    decode = Decoder(layers, a.width)
    ms, _ = timed(lambda: decode(tokens[:1]), 200)
    print(f"decoding: {ms * 1e3:.1f} us a token, {2 * a.layers * a.width * a.hidden / ms * 1e-9:.2f} TB/s of weights")
    status = ap.ap_check()
    if status:
        raise ap.APError(status, "ap_check")


if __name__ == "__main__":
    main()

"""Cases that measure the 8-bit block-scaled operators: the root-mean-square
norm with the residual's addition and its gradient, the quantiser to e4m3 with
a scale for each block of 128, and the matrix product over such operands.

``prepare`` makes what a program holds before the call, ``run`` makes one pass
(in plain 32-bit torch operations, or through the library where ``own`` is
true), ``exact`` gives the same outputs from the definitions in 64 bits, and
``work`` counts the bytes and operations a pass cannot do without.

The definitions. A block is 128 consecutive values of a row (the last one of a
row may be shorter), or a 128 x 128 tile. Its scale is
``s = max(amax|block| / 448, 2^-126)`` and a value v is held as
``e4m3(v * (1 / s))``; 448 is e4m3's largest value.

* norm: ``h = x + residual``; ``rstd = 1 / sqrt(mean(h^2) + eps)`` over a row;
  ``y = h * rstd * weight``, written in the input's type and / or as e4m3 with
  a scale for each block of a row. ``h`` is written back as the new residual.
* norm gradient: with ``n = h * rstd`` and ``g = dy * weight``,
  ``dx = rstd * (g - n * mean(g * n)) + dresidual`` and
  ``dweight = sum over rows of dy * n``.
* quantize: e4m3 and scales of a matrix, by row blocks or by tiles, and / or of
  its transpose.
* matmul: ``c[i, j] = sum_k a[i, k] sa[i, k / 128] b[j, k] sb``, where sb is a
  scale of a 128 x 128 tile of b (a weight) or of a row block of b.
"""

import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -126
BLOCK = 128
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def blocks(n):
    return (n + BLOCK - 1) // BLOCK


def padded(n):
    """Leading dimension of a row of n bytes: rows of 8-bit operands start on 16-byte boundaries."""
    return (n + 15) // 16 * 16


def listed():
    return [
        # one token of a decode step through a pre-norm layer of 4096 channels
        {"name": "norm 1x4096", "op": "norm", "rows": 1, "cols": 4096, "type": "bf16", "residual": "same", "out": "q"},
        # a ragged prompt batch, a width that is no multiple of the block, no residual, both outputs
        {"name": "norm 1237x5000 f16", "op": "norm", "rows": 1237, "cols": 5000, "type": "f16", "residual": "none", "out": "both"},
        # a training batch with the residual stream kept in 32 bits
        {"name": "norm 32768x8192 f32 residual", "op": "norm", "rows": 32768, "cols": 8192, "type": "bf16", "residual": "f32", "out": "q"},
        # the norm's gradient for a small batch in 32 bits, and for a training batch
        {"name": "norm grad 777x2560 f32", "op": "norm_grad", "rows": 777, "cols": 2560, "type": "f32", "residual": "same", "dresidual": False},
        {"name": "norm grad 16384x8192", "op": "norm_grad", "rows": 16384, "cols": 8192, "type": "bf16", "residual": "same", "dresidual": True},
        # activations of 64 decoding sequences before a wide projection
        {"name": "quantize 64x16384", "op": "quantize", "rows": 64, "cols": 16384, "type": "bf16", "block": 1, "out": "rows"},
        # an output gradient of a training batch: rows for the input's gradient, columns for the weight's
        {"name": "quantize 16384x8192 both", "op": "quantize", "rows": 16384, "cols": 8192, "type": "bf16", "block": 1, "out": "both"},
        # a 32-bit master weight with odd sizes, by tiles, with its transpose for the backward product
        {"name": "quantize weight 11003x4100", "op": "quantize", "rows": 11003, "cols": 4100, "type": "f32", "block": 128, "out": "both"},
        # one token times a square weight: the weight is read once
        {"name": "matmul 1x8192x8192", "op": "matmul", "m": 1, "n": 8192, "k": 8192, "b_block": 128, "type": "bf16"},
        # a ragged prompt times a weight of odd sizes
        {"name": "matmul 333x4104x5000", "op": "matmul", "m": 333, "n": 4104, "k": 5000, "b_block": 128, "type": "f16"},
        # a training batch's forward product
        {"name": "matmul 8192x8192x8192", "op": "matmul", "m": 8192, "n": 8192, "k": 8192, "b_block": 128, "type": "bf16"},
        # a weight gradient: both operands are activations scaled by row blocks, the result in 32 bits
        {"name": "matmul grad 4096x8192x16384", "op": "matmul", "m": 4096, "n": 8192, "k": 16384, "b_block": 1, "type": "f32"},
    ]


def spread(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "quantize", "matmul"])
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "matmul":
        if rng.random() < 0.5:  # serving: few tokens, a large weight
            m, n, k = spread(rng, 1, 128), spread(rng, 256, 16384), spread(rng, 256, 16384)
        else:
            m, n = spread(rng, 128, 8192), spread(rng, 128, 8192)
            k = spread(rng, 128, min(16384, 2 ** 39 // (m * n)))
        return {"op": op, "m": m, "n": n, "k": k, "b_block": rng.choice([1, 128]), "type": kind}
    cols = spread(rng, 64, 16384)
    rows = spread(rng, 1, min(32768, 2 ** 28 // cols))
    if op == "quantize":
        return {"op": op, "rows": rows, "cols": cols, "type": kind, "block": rng.choice([1, 128]),
                "out": rng.choice(["rows", "cols", "both"])}
    residual = rng.choice(["same", "f32"])
    if op == "norm_grad":
        return {"op": op, "rows": rows, "cols": cols, "type": kind, "residual": residual, "dresidual": rng.random() < 0.5}
    return {"op": op, "rows": rows, "cols": cols, "type": kind, "residual": rng.choice([residual, "none"]),
            "out": rng.choice(["q", "y", "both"])}


def residual_type(case):
    return TYPES[case["type"]] if case["residual"] == "same" else torch.float32


def empty8(rows, cols):
    """Room for rows of e4m3 values that start on 16-byte boundaries."""
    return torch.empty(rows, padded(cols), dtype=torch.uint8, device="cuda").view(E4M3)[:, :cols]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def channels(n):  # activations: a few channels are many times larger than the rest
        return torch.exp(0.5 * normal(n)) * (1 + 20 * (torch.rand(n, generator=gen, device="cuda") < 0.002))

    state = {"case": case}
    f32 = dict(dtype=torch.float32, device="cuda")
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        a, b = normal(m, k).mul_(channels(k)), normal(n, k).mul_(k ** -0.5)
        for name, v, block in (("a", a, 1), ("b", b, case["b_block"])):
            q, s = quantized(v, block)
            state[name] = empty8(*v.shape)
            state[name].view(torch.uint8).copy_(q.view(torch.uint8))
            state[name + "_scales"] = s
        state["c"] = torch.empty(m, n, dtype=TYPES[case["type"]], device="cuda")
        return state
    rows, cols, kind = case["rows"], case["cols"], TYPES[case["type"]]
    if case["op"] == "quantize":
        state["x"] = (normal(rows, cols).mul_(channels(cols)) * (0.02 if case["block"] == 128 else 1.0)).to(kind)
        state["q"] = state["scales"] = state["qt"] = state["scales_t"] = None
        by_tile = case["block"] == 128
        if case["out"] != "cols":
            state["q"] = empty8(rows, cols)
            state["scales"] = torch.empty(blocks(rows) if by_tile else rows, blocks(cols), **f32)
        if case["out"] != "rows":
            state["qt"] = empty8(cols, rows)
            state["scales_t"] = torch.empty(blocks(cols) if by_tile else cols, blocks(rows), **f32)
        return state
    state["weight"] = 1 + 0.1 * normal(cols)
    if case["op"] == "norm_grad":
        rt = residual_type(case)
        h = normal(rows, cols).mul_(channels(cols))
        state["rstd"] = 1 / torch.sqrt(h.square().mean(1) + EPS)
        state["h"] = h.to(rt)
        state["dy"] = (1e-3 * normal(rows, cols)).to(kind)
        state["dresidual"] = (1e-3 * normal(rows, cols)).to(rt) if case["dresidual"] else None
        state["dx"] = torch.empty(rows, cols, dtype=rt, device="cuda")
        state["dweight"] = torch.empty(cols, **f32)
        return state
    state["x"] = normal(rows, cols).mul_(channels(cols)).to(kind)
    state["residual"] = state["h"] = state["y"] = state["q"] = state["scales"] = None
    if case["residual"] != "none":
        state["residual"] = normal(rows, cols).mul_(2).to(residual_type(case))
        state["h"] = torch.empty_like(state["residual"])
    if case["out"] != "q":
        state["y"] = torch.empty(rows, cols, dtype=kind, device="cuda")
    if case["out"] != "y":
        state["q"] = empty8(rows, cols)
        state["scales"] = torch.empty(rows, blocks(cols), **f32)
    state["rstd"] = torch.empty(rows, **f32)
    return state


# ------------------------------------------------------------------ plain form


def in_blocks(v, block):
    """v padded with zeros to whole blocks: [row blocks, block, column blocks, 128]."""
    rows, cols = v.shape
    v = torch.nn.functional.pad(v, (0, -cols % BLOCK, 0, -rows % block))
    return v.view(-1, block, blocks(cols), BLOCK)


def quantized(v, block):
    """e4m3 values and scales of a 32-bit matrix by row blocks (1) or tiles (128)."""
    w = in_blocks(v, block)
    s = (w.abs().amax((1, 3), keepdim=True) / E4M3_MAX).clamp(min=MIN_SCALE)
    q = (w * (1 / s)).to(E4M3)
    return q.view(w.shape[0] * block, -1)[: v.shape[0], : v.shape[1]], s.view(w.shape[0], -1)


def expanded(s, rows, cols, block):
    return s.repeat_interleave(block, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :cols]


def plain_norm(state):
    case = state["case"]
    h = state["x"].float()
    out = {}
    if state["residual"] is not None:
        h = h + state["residual"].float()
        out["h"] = h.to(state["residual"].dtype)
    out["rstd"] = 1 / torch.sqrt(h.square().mean(1) + EPS)
    y = h * out["rstd"][:, None] * state["weight"]
    if case["out"] != "q":
        out["y"] = y.to(state["x"].dtype)
    if case["out"] != "y":
        out["q"], out["scales"] = quantized(y, 1)
    return out


def plain_norm_grad(state):
    dy, n = state["dy"].float(), state["h"].float() * state["rstd"][:, None]
    g = dy * state["weight"]
    dx = state["rstd"][:, None] * (g - n * (g * n).mean(1, keepdim=True))
    if state["dresidual"] is not None:
        dx = dx + state["dresidual"].float()
    return {"dx": dx.to(state["h"].dtype), "dweight": (dy * n).sum(0)}


def plain_quantize(state):
    x, block, out = state["x"].float(), state["case"]["block"], {}
    if state["q"] is not None:
        out["q"], out["scales"] = quantized(x, block)
    if state["qt"] is not None:
        out["qt"], out["scales_t"] = quantized(x.t().contiguous(), block)
    return out


def plain_matmul(state):
    a, b = state["a"], state["b"]
    a = a.float() * expanded(state["a_scales"], *a.shape, 1)
    b = b.float() * expanded(state["b_scales"], *b.shape, state["case"]["b_block"])
    return {"c": (a @ b.t()).to(state["c"].dtype)}


# ------------------------------------------------------------------ the library's calls


def own_norm(state):
    import async_global_shared_gb300 as ap

    ap.ap_rms_norm(state["x"], state["weight"], EPS, y=state["y"], q=state["q"], q_scales=state["scales"],
                   residual=state["residual"], residual_out=state["h"], rstd=state["rstd"])
    return {k: state[k] for k in ("h", "rstd", "y", "q", "scales") if state[k] is not None}


def own_norm_grad(state):
    import async_global_shared_gb300 as ap

    if "workspace" not in state:  # kept by a training program for as long as its sizes stay
        size = ap.ap_rms_norm_backward_workspace(*state["dy"].shape)
        state["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    ap.ap_rms_norm_backward(state["dy"], state["h"], state["weight"], state["rstd"], state["dx"], state["dweight"],
                            state["workspace"], dresidual=state["dresidual"])
    return {"dx": state["dx"], "dweight": state["dweight"]}


def own_quantize(state):
    import async_global_shared_gb300 as ap

    ap.ap_quantize(state["x"], state["case"]["block"], q=state["q"], scales=state["scales"], qt=state["qt"],
                   scales_t=state["scales_t"])
    return {k: state[k] for k in ("q", "scales", "qt", "scales_t") if state[k] is not None}


def own_matmul(state):
    import async_global_shared_gb300 as ap

    ap.ap_matmul_fp8(state["a"], state["a_scales"], state["b"], state["b_scales"], state["c"], state["case"]["b_block"])
    return {"c": state["c"]}


PLAIN = {"norm": plain_norm, "norm_grad": plain_norm_grad, "quantize": plain_quantize, "matmul": plain_matmul}
OWN = {"norm": own_norm, "norm_grad": own_norm_grad, "quantize": own_quantize, "matmul": own_matmul}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------ 64 bits


def exact_quantized(v, block):
    """v / s before its rounding to e4m3, and s, in 64 bits: every block's amax, then one division."""
    rows, cols = v.shape
    s = torch.zeros(-(-rows // block), blocks(cols), dtype=torch.float64, device=v.device)
    r = torch.arange(rows, device=v.device) // block
    tall = torch.zeros(s.shape[0], cols, dtype=torch.float64, device=v.device)
    tall.index_reduce_(0, r, v.abs(), "amax", include_self=True)
    for j in range(s.shape[1]):
        s[:, j] = tall[:, j * BLOCK:(j + 1) * BLOCK].amax(1) / E4M3_MAX
    s.clamp_(min=MIN_SCALE)
    q = torch.empty_like(v)
    for j in range(s.shape[1]):
        q[:, j * BLOCK:(j + 1) * BLOCK] = v[:, j * BLOCK:(j + 1) * BLOCK] / s[r, j][:, None]
    return q, s


def exact(case, seed):
    state = prepare(case, seed)
    d = {k: v.double() for k, v in state.items() if isinstance(v, torch.Tensor)}
    if case["op"] == "matmul":
        c = torch.zeros_like(d["c"])
        for j in range(blocks(case["k"])):  # one block of the sum at a time
            at = slice(j * BLOCK, (j + 1) * BLOCK)
            sb = d["b_scales"][:, j].repeat_interleave(case["b_block"])[: case["n"]]
            c += torch.einsum("ik,jk->ij", d["a"][:, at], d["b"][:, at]) * torch.outer(d["a_scales"][:, j], sb)
        return {"c": c}
    if case["op"] == "quantize":
        out = {}
        if case["out"] != "cols":
            out["q"], out["scales"] = exact_quantized(d["x"], case["block"])
        if case["out"] != "rows":
            out["qt"], out["scales_t"] = exact_quantized(d["x"].T, case["block"])
        return out
    if case["op"] == "norm_grad":
        # the gradient of sum(dy * y) with respect to h, with rstd's own
        # dependence on h written out: d rstd / d h_i = -rstd^3 h_i / cols
        h, r, w, dy = d["h"], d["rstd"][:, None], d["weight"], d["dy"]
        along = torch.einsum("ij,j,ij->i", dy, w, h)[:, None] / case["cols"]
        dx = torch.addcmul(dy * w * r, h, along * r ** 3, value=-1)
        return {"dx": dx + d["dresidual"] if "dresidual" in d else dx, "dweight": torch.einsum("ij,ij,i->j", dy, h, d["rstd"])}
    h = torch.add(d["x"], d["residual"]) if "residual" in d else d["x"]
    rstd = torch.rsqrt(torch.einsum("ij,ij->i", h, h) / case["cols"] + EPS)
    y = torch.einsum("ij,i,j->ij", h, rstd, d["weight"])
    out = {"rstd": rstd}
    if "residual" in d:
        out["h"] = h
    if case["out"] != "q":
        out["y"] = y
    if case["out"] != "y":
        out["q"], out["scales"] = exact_quantized(y, 1)
    return out


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        scales = m * blocks(k) + (n if case["b_block"] == 1 else blocks(n)) * blocks(k)
        return {"bytes": m * k + n * k + 4 * scales + TYPES[case["type"]].itemsize * m * n, "flops": 2 * m * n * k}
    rows, cols, size = case["rows"], case["cols"], TYPES[case["type"]].itemsize
    n = rows * cols
    if case["op"] == "quantize":
        each = n + 4 * (n // BLOCK if case["block"] == 1 else n // BLOCK ** 2)
        return {"bytes": n * size + each * (2 if case["out"] == "both" else 1), "flops": 3 * n}
    if case["op"] == "norm_grad":
        rt = residual_type(case).itemsize
        return {"bytes": n * (size + rt * (3 if case["dresidual"] else 2)) + 4 * rows + 8 * cols, "flops": 9 * n}
    moved = n * size + 4 * rows + 4 * cols
    if case["residual"] != "none":
        moved += 2 * n * residual_type(case).itemsize
    if case["out"] != "q":
        moved += n * size
    if case["out"] != "y":
        moved += n + 4 * rows * blocks(cols)
    return {"bytes": moved, "flops": 7 * n}

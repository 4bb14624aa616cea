"""Cases of the operators of an expert layer in 8-bit floating point and in training, with their plain forms.

They stand around dispatch and combine, as the router and the int8 products do:

  norm            rows (and the residual to add) -> root-mean-square norm, as rows or as E4M3 codes with a
                  scale for each 128 channels (what a pre-quantised dispatch takes), and the residual's sum
  norm_backward   gradient of the norm -> gradient of the rows and of the weight
  quantize        rows -> E4M3 codes with a scale for each 128 channels
  product         E4M3 rows times E4M3 weights (one matrix, or one for each expert's rows) with scales for
                  128 channels of a row and 128 x 128 of a weight, with an optional SwiGLU epilogue
  block           16-bit rows times 16-bit weights, as a rule gate and up projection with SwiGLU
  block_backward  its gradients: of the rows, and of the weights

``run`` computes them from elementary torch operations, or, with ``own`` set, through the package's public
calls.  ``exact`` is a second computation in 64 bits.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
E4M3 = torch.float8_e4m3fn
EPS = 1e-6
ALIGN = 16  # rows of an expert start at multiples of this, as the layout's expert_alignment makes them


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------

def _norm(name, rows, cols, dtype, residual=True, fp8=False, keep=True):
    return dict(name=name, op="norm", rows=rows, cols=cols, dtype=dtype, residual=residual, fp8=fp8, keep=keep)


def _norm_backward(name, rows, cols, dtype, through=True):
    return dict(name=name, op="norm_backward", rows=rows, cols=cols, dtype=dtype, through=through)


def _quant(name, rows, cols, dtype):
    return dict(name=name, op="quantize", rows=rows, cols=cols, dtype=dtype)


def _rows(name, op, rows, inner, outer, groups, gated, dtype="bf16", skew=0.5, col_major=False):
    return dict(name=name, op=op, rows=rows, inner=inner, outer=outer, groups=groups, gated=gated, dtype=dtype,
                skew=skew, col_major=col_major)


def listed():
    return [
        # one token of a serving step in front of an expert layer: rows for the router, codes for dispatch
        _norm("norm one token", 1, 7168, "bf16", fp8=True),
        # a prefill batch of 8 ranks x 4096 tokens, the same
        _norm("norm prefill", 32768, 7168, "bf16", fp8=True),
        # a ragged small batch in training, fp32
        _norm_backward("norm gradient ragged", 1003, 4096, "fp32", through=False),
        # the forward+backward step's tokens, with the residual's gradient passing through
        _norm_backward("norm gradient training", 262144, 4096, "bf16"),
        # activations of a decode step before the down projection
        _quant("quantize decode rows", 96, 2048, "bf16"),
        # activations of an expanded prefill batch before the down projection
        _quant("quantize prefill rows", 65536, 2048, "bf16"),
        # a shared expert's gate and up projection on one token
        _rows("fp8 product one token", "product", 1, 7168, 4096, 0, True),
        # one rank's 32 local experts in a decode step: 2 to 4 rows each, some experts empty
        _rows("fp8 product decode experts", "product", 96, 7168, 4096, 32, True),
        # gate and up projection of 64 local experts on a large expanded batch, scales as dispatch lays them out by columns
        _rows("fp8 product prefill gate up", "product", 65536, 7168, 4096, 64, True, skew=0.1, col_major=True),
        # a shared expert in 16 bits on one token
        _rows("block one token", "block", 1, 7168, 4096, 0, True),
        # gate and up projection of 32 local experts in a training step
        _rows("block training", "block", 65536, 4096, 4096, 32, True, skew=0.1),
        # its backward pass: rows and weights
        _rows("block training gradient", "block_backward", 65536, 4096, 4096, 32, True, skew=0.1),
    ]


def _spread(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "quantize", "product", "product", "block", "block",
                     "block_backward", "block_backward"])
    if op in ("norm", "norm_backward", "quantize"):
        c = dict(op=op, rows=_spread(rng, 1, 131072), cols=_spread(rng, 48, 8192),
                 dtype=rng.choice(["bf16", "fp16", "fp32"]))
        if rng.random() < 0.7:
            c["cols"] = max(128, c["cols"] // 128 * 128)
        if op == "norm":
            c.update(residual=rng.random() < 0.7, fp8=rng.random() < 0.5)
            c["keep"] = not c["fp8"] or rng.random() < 0.5
        elif op == "norm_backward":
            c.update(through=rng.random() < 0.5)
        return c
    groups = rng.choice([0, 1, 8, 64, _spread(rng, 1, 64)])
    gated = rng.random() < 0.6
    c = dict(op=op, rows=_spread(rng, 1, 32768), groups=groups, gated=gated, skew=rng.choice([0.0, 0.1, 0.5]),
             col_major=op == "product" and rng.random() < 0.5)
    if op == "product":
        c.update(inner=16 * _spread(rng, 8, 448), outer=(2 if gated else 1) * _spread(rng, 32, 2048),
                 dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    elif op == "block":
        c.update(inner=8 * _spread(rng, 8, 896), outer=(2 if gated else 1) * _spread(rng, 32, 2048),
                 dtype=rng.choice(["bf16", "bf16", "fp16"]))
    else:
        c.update(inner=8 * _spread(rng, 8, 512), outer=(16 if gated else 8) * _spread(rng, 4, 256),
                 dtype=rng.choice(["bf16", "bf16", "fp16"]))
    return c


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _codes(g, *shape):
    """E4M3 codes of normal values whose block maximum is near four deviations."""
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float16).mul_(112).clamp_(-448, 448).to(E4M3).view(torch.uint8)


def _row_counts(case, seed):
    """Rows of each expert: a draw over skewed popularities, so that some experts stay empty."""
    r = np.random.default_rng([seed, 7])
    p = 1.0 / (1.0 + r.permutation(case["groups"])) ** case["skew"]
    return r.multinomial(case["rows"], p / p.sum())


def _blocks(n):
    return (n + 127) // 128


def _activations(g, rows, cols):
    """Rows of different sizes, a few channels far above the rest, as activations have them."""
    x = _randn(g, rows, cols) * torch.exp(0.5 * _randn(g, rows, 1))
    x[:, :: 61] *= 6
    return x


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    t = TYPES[case["dtype"]]
    if op in ("norm", "norm_backward", "quantize"):
        N, H = case["rows"], case["cols"]
        s["x"] = _activations(g, N, H).to(t)
        if op != "quantize":
            s["weight"] = (1 + 0.1 * _randn(g, H)).to(t)
        if op == "norm":
            s["residual"] = _activations(g, N, H).to(t) if case["residual"] else None
        elif op == "norm_backward":
            s["grad"] = _randn(g, N, H).to(t)
            s["through"] = _randn(g, N, H).to(t) if case["through"] else None
        return s
    G, inner, outer, gated = case["groups"], case["inner"], case["outer"], case["gated"]
    M = case["rows"] + G * (ALIGN - 1)  # room for every expert's padding
    width = outer // 2 if gated else outer
    wshape = (G, outer, inner) if G else (outer, inner)
    if op == "product":
        s["a"] = _codes(g, M, inner)
        scales = (_blocks(inner), M) if case["col_major"] else (M, _blocks(inner))
        s["a_scale"] = (torch.rand(scales, generator=g, device=DEV) + 0.5) * (4 / 448)
        s["w"] = _codes(g, *wshape)
        # the blocks of 128 channels start anew at the up projection
        nb = 2 * _blocks(width) if gated else _blocks(outer)
        s["w_scale"] = (torch.rand(wshape[:-2] + (nb, _blocks(inner)), generator=g, device=DEV) + 0.5) * (4 / 448 / math.sqrt(inner))
    else:
        s["a"] = _randn(g, M, inner).to(t)
        s["w"] = torch.randn(wshape, generator=g, device=DEV, dtype=torch.float16).mul_(1 / math.sqrt(inner)).to(t)
        if op == "block_backward":
            s["grad"] = _randn(g, M, width).to(t)
            # what the forward pass kept: the projections before the gate
            s["pre"] = _randn(g, M, outer).to(t) if gated else None
    s["out"] = torch.zeros((M, inner if op == "block_backward" else width), dtype=t, device=DEV)
    if G:
        n = _row_counts(case, seed)
        start = np.concatenate([[0], np.cumsum((n + ALIGN - 1) // ALIGN * ALIGN)])[:-1]
        s["most"] = int(n.max())
        s["start"] = torch.from_numpy(start.astype(np.int64)).to(DEV)
        s["count"] = torch.from_numpy(n.astype(np.int32)).to(DEV)
    return s


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------

def run(state):
    c = state["case"]
    if own:
        return _call(c, state)
    return {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "quantize": _plain_quantize,
            "product": _plain_product, "block": _plain_block, "block_backward": _plain_block_backward}[c["op"]](c, state)


def _call(c, s):
    import combine_topk_idx_expert_amd as ep

    if c["op"] == "norm":
        y, q, total = ep.rms_norm(s["x"], s["weight"], eps=EPS, residual=s["residual"], fp8=c["fp8"], keep=c["keep"])
        return y, (q[0].view(E4M3), q[1]) if c["fp8"] else None, total
    if c["op"] == "norm_backward":
        return ep.rms_norm_backward(s["x"], s["weight"], s["grad"], eps=EPS, grad_total=s["through"])
    if c["op"] == "quantize":
        codes, scales = ep.quantize_fp8(s["x"])
        return codes.view(E4M3), scales
    rows = (s["start"], s["count"]) if c["groups"] else None
    if c["op"] == "product":
        return ep.matmul_fp8((s["a"], s["a_scale"]), (s["w"], s["w_scale"]), rows=rows, gated=c["gated"],
                             scales_col_major=c["col_major"], out=s["out"])
    if c["op"] == "block":
        return ep.matmul(s["a"], s["w"], rows=rows, gated=c["gated"], out=s["out"])
    return ep.matmul_backward(s["a"], s["w"], s["grad"], rows=rows, gated=c["gated"], pre=s["pre"],
                              out=(s["out"], torch.empty_like(s["w"])))


def _quantized(x):
    """Codes and scales of fp32 rows, blocks of 128 channels, the last one shorter where they do not come out."""
    N, H = x.shape
    b = torch.nn.functional.pad(x, (0, _blocks(H) * 128 - H)).view(N, _blocks(H), 128)
    scale = b.abs().amax(2) / 448
    q = torch.where(scale[:, :, None] > 0, b / scale[:, :, None], b)
    return q.reshape(N, -1)[:, :H].to(E4M3), scale


def _plain_norm(c, s):
    t = s["x"].dtype
    x = s["x"].float()
    if s["residual"] is not None:
        x = x + s["residual"].float()
    y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * s["weight"].float()
    return (y.to(t) if c["keep"] else None, _quantized(y) if c["fp8"] else None,
            x.to(t) if s["residual"] is not None else None)


def _plain_norm_backward(c, s):
    x, w, g = s["x"].float(), s["weight"].float(), s["grad"].float()
    r = torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
    n = x * r
    gw = g * w
    d = r * (gw - n * (gw * n).mean(1, keepdim=True))
    if s["through"] is not None:
        d = d + s["through"].float()
    # the sum over all rows is a long one
    return d.to(s["x"].dtype), (g * n).sum(0, dtype=torch.float64).float()


def _plain_quantize(c, s):
    return _quantized(s["x"].float())


def _gather(c, s):
    """Rows of one expert side by side, as many as the fullest has: their indices, and which of them are."""
    lane = torch.arange(max(s["most"], 1), device=DEV)
    there = lane < s["count"][:, None]
    return torch.where(there, s["start"][:, None] + lane, 0), there


def _weights(s):
    """E4M3 weights as fp32, their scales applied."""
    w, ws = s["w"].view(E4M3).float(), s["w_scale"]
    outer, inner = w.shape[-2:]
    if s["case"]["gated"]:  # the blocks start anew at the second half
        at = torch.arange(outer // 2, device=DEV) // 128
        at = torch.cat([at, at + ws.shape[-2] // 2])
    else:
        at = torch.arange(outer, device=DEV) // 128
    return w * ws[..., at, :][..., torch.arange(inner, device=DEV) // 128]


def _times(c, s, x, w):
    """fp32 rows times fp32 weights [.., outer, inner], and the gate."""
    if c["groups"]:
        at, there = _gather(c, s)
        y = torch.bmm(w, x[at].transpose(1, 2).contiguous()).transpose(1, 2)  # [G, most, outer]
    else:
        y = x @ w.t()
    if c["gated"]:
        gate, up = y.chunk(2, dim=-1)
        y = gate * torch.sigmoid(gate) * up
    y = y.to(s["out"].dtype)
    if c["groups"]:
        s["out"][at[there]] = y[there]
        return s["out"]
    return y


def _plain_product(c, s):
    scale = s["a_scale"].t() if c["col_major"] else s["a_scale"]
    x = s["a"].view(E4M3).float() * scale[:, torch.arange(c["inner"], device=DEV) // 128]
    return _times(c, s, x, _weights(s))


def _plain_block(c, s):
    return _times(c, s, s["a"].float(), s["w"].float())


def _plain_block_backward(c, s):
    x, w, d = s["a"].float(), s["w"].float(), s["grad"].float()
    if c["gated"]:
        gate, up = s["pre"].float().chunk(2, dim=1)
        p = torch.sigmoid(gate)
        d = torch.cat([d * up * p * (1 + gate * (1 - p)), d * gate * p], 1)
    t = s["a"].dtype
    if not c["groups"]:
        return (d @ w).to(t), (d.t() @ x).to(t)
    at, there = _gather(c, s)
    d = torch.where(there[:, :, None], d[at], 0.0)  # [G, most, outer]
    gx = torch.bmm(d, w)
    s["out"][at[there]] = gx[there].to(t)
    del gx
    return s["out"], torch.bmm(d.transpose(1, 2).contiguous(), x[at]).to(t)


# ------------------------------------------------------------------------------------------
# what a pass cannot do without, and the values in 64 bits
# ------------------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    size = 4 if case["dtype"] == "fp32" else 2
    if op in ("norm", "norm_backward", "quantize"):
        n = case["rows"] * case["cols"]
        coded = n + case["rows"] * _blocks(case["cols"]) * 4
        if op == "quantize":
            return {"bytes": n * size + coded, "flops": n * 2}
        if op == "norm":
            return {"bytes": n * size * (1 + 2 * case["residual"] + case["keep"]) + coded * case["fp8"] + case["cols"] * size,
                    "flops": n * 5}
        return {"bytes": n * size * (3 + case["through"]) + case["cols"] * (size + 4), "flops": n * 10}
    G, M, inner, outer, gated = case["groups"], case["rows"], case["inner"], case["outer"], case["gated"]
    width = outer // 2 if gated else outer
    experts = min(G, M) if G else 1
    if op == "product":
        return {"bytes": M * (inner + _blocks(inner) * 4) + experts * outer * inner + M * width * size,
                "flops": 2 * M * inner * outer}
    if op == "block":
        return {"bytes": (M * inner + experts * outer * inner + M * width) * size, "flops": 2 * M * inner * outer}
    # weights read for the experts that have rows; their gradients are written for all
    return {"bytes": (2 * M * inner + M * width + (M * outer if gated else 0)
                      + (experts + max(G, 1)) * outer * inner) * size,
            "flops": 4 * M * inner * outer}


def _exact_quantized(y):
    """The values that codes stand for follow from the scales; a value near the border of two codes has no one code."""
    N, H = y.shape
    scale = torch.stack([y[:, i:i + 128].abs().amax(1) for i in range(0, H, 128)], 1) / 448
    return None, scale


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_quantized(s["x"].double())
    if op == "norm":
        x = s["x"].double()
        if s["residual"] is not None:
            x += s["residual"].double()
        y = x / torch.sqrt(torch.linalg.vector_norm(x, dim=1, keepdim=True) ** 2 / x.shape[1] + EPS) * s["weight"].double()
        return (y if case["keep"] else None, _exact_quantized(y) if case["fp8"] else None,
                x if s["residual"] is not None else None)
    if op == "norm_backward":
        w = s["weight"].double()
        grad_x, grad_w = [], torch.zeros_like(w)
        for i in range(0, case["rows"], 16384):  # rows are independent, and 64 bits of all of them are many
            x, g = s["x"][i:i + 16384].double(), s["grad"][i:i + 16384].double()
            inv = 1 / torch.sqrt((x * x).sum(1, keepdim=True) / case["cols"] + EPS)
            dot = (g * w * x).sum(1, keepdim=True)
            d = inv * g * w - x * inv ** 3 * dot / case["cols"]
            if s["through"] is not None:
                d += s["through"][i:i + 16384].double()
            grad_x.append(d)
            grad_w += (g * x * inv).sum(0)
        return torch.cat(grad_x), grad_w
    G, outer, inner, gated = case["groups"], case["outer"], case["inner"], case["gated"]
    starts = s["start"].tolist() if G else [0]
    counts = s["count"].tolist() if G else [case["rows"]]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    grad_w = torch.zeros(s["w"].shape, dtype=torch.float64, device=DEV) if op == "block_backward" else None
    for e, (lo, n) in enumerate(zip(starts, counts)):
        if n == 0:
            continue
        a, w = s["a"][lo:lo + n], s["w"][e] if G else s["w"]
        if op == "product":
            sa = s["a_scale"].t()[lo:lo + n] if case["col_major"] else s["a_scale"][lo:lo + n]
            sw = (s["w_scale"][e] if G else s["w_scale"]).double()
            if gated:
                half = sw.shape[0] // 2
                sw = torch.cat([v.repeat_interleave(128, 0)[: outer // 2] for v in (sw[:half], sw[half:])])
            else:
                sw = sw.repeat_interleave(128, 0)[:outer]
            a = a.view(E4M3).double() * sa.double().repeat_interleave(128, 1)[:, :inner]
            w = w.view(E4M3).double() * sw.repeat_interleave(128, 1)[:, :inner]
        else:
            a, w = a.double(), w.double()
        if op == "block_backward":
            d = s["grad"][lo:lo + n].double()
            if gated:
                pre = s["pre"][lo:lo + n].double().requires_grad_()
                y = torch.nn.functional.silu(pre[:, : outer // 2]) * pre[:, outer // 2:]
                (d,) = torch.autograd.grad(y, pre, d)
            out[lo:lo + n] = d @ w
            (grad_w[e] if G else grad_w).copy_(d.t() @ a)
            continue
        y = torch.nn.functional.linear(a, w)
        if gated:
            y = y[:, : outer // 2] / (1 + torch.exp(-y[:, : outer // 2])) * y[:, outer // 2:]
        out[lo:lo + n] = y
    return (out, grad_w) if op == "block_backward" else out

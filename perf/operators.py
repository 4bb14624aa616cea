"""Cases of the routing and 8-bit integer product operators, with their plain forms.

Four operators stand around dispatch and combine:

  route           router logits -> topk_idx and topk_weights, what the layout and combine take
  route_backward  gradient of topk_weights -> gradient of the logits
  quantize        rows -> int8 codes and one fp32 scale a row
  product         int8 rows times the int8 weights of their expert (or of one dense layer),
                  scaled for each token and output channel, with an optional SwiGLU epilogue

``run`` computes them from elementary torch operations, or, with ``own`` set, through the
package's public calls.  ``exact`` is a second computation in 64 bits.
"""

from __future__ import annotations

import functools
import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
ALIGN = 16  # rows of an expert start at multiples of this, as the layout's expert_alignment makes them


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------

def _route(name, T, E, K, score, dtype, bias=False, groups=1, top_groups=1, group_score="max", renorm=True,
           scale=1.0, masked=0.0, op="route"):
    return dict(name=name, op=op, T=T, E=E, K=K, score=score, dtype=dtype, bias=bias, groups=groups,
                top_groups=top_groups, group_score=group_score, renorm=renorm, scale=scale, masked=masked)


def _quant(name, rows, cols, dtype):
    return dict(name=name, op="quantize", rows=rows, cols=cols, dtype=dtype)


def _product(name, rows, inner, outer, groups, gated, dtype="bf16", skew=0.5):
    return dict(name=name, op="product", rows=rows, inner=inner, outer=outer, groups=groups, gated=gated,
                dtype=dtype, skew=skew)


def listed():
    return [
        # one token of a serving step: 256 experts, 4 of 8 groups by the sum of their two best, balance bias
        _route("route one token", 1, 256, 8, "sigmoid", "fp32", bias=True, groups=8, top_groups=4,
               group_score="top2", scale=2.5),
        # a padded prefill batch of 8 ranks x 4096 tokens, softmax over the chosen experts
        _route("route prefill", 32768, 256, 8, "softmax", "bf16", masked=0.05),
        # the forward+backward step's routing: 32 ranks x 8192 tokens
        _route("route training step", 262144, 256, 8, "sigmoid", "fp32", bias=True, groups=8, top_groups=4,
               group_score="top2", scale=2.5),
        # its gradient: only the chosen experts' logits get one, the rest of the row is zero
        _route("route gradient", 262144, 256, 8, "sigmoid", "fp32", bias=True, groups=8, top_groups=4,
               group_score="top2", scale=2.5, op="route_backward"),
        # softmax over all experts without renormalising (a dense gradient), 128 ranks x 1024 tokens, top 6
        _route("route gradient dense", 131072, 256, 6, "softmax", "bf16", renorm=False, op="route_backward"),
        # the expanded rows of a small serving batch
        _quant("quantize decode rows", 129, 7168, "bf16"),
        # the tokens of the forward+backward step before dispatch
        _quant("quantize training rows", 262144, 4096, "bf16"),
        # a shared expert's gate and up projection on one token
        _product("product one token", 1, 7168, 4096, 0, True),
        # one rank's 32 local experts in a decode step: 2 to 4 rows each, some experts empty
        _product("product decode experts", 96, 7168, 4096, 32, True),
        # a dense down projection on a ragged batch
        _product("product dense ragged", 1003, 2048, 7168, 0, False),
        # down projection of 64 local experts on an expanded prefill batch
        _product("product prefill down", 16384, 2048, 7168, 64, False, skew=0.1),
        # gate and up projection of 64 local experts on a large expanded batch
        _product("product prefill gate up", 65536, 7168, 4096, 64, True, skew=0.1),
    ]


def _spread(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["route", "route", "route_backward", "quantize", "product", "product", "product"])
    if op in ("route", "route_backward"):
        groups = rng.choice([1, 1, 4, 8])
        E = groups * _spread(rng, 8, 512 // groups)
        top_groups = rng.randint(1, groups)
        score = rng.choice(["softmax", "sigmoid"])
        return dict(op=op, T=_spread(rng, 1, 131072), E=E, K=rng.randint(1, min(10, top_groups * (E // groups))),
                    score=score, dtype=rng.choice(["fp32", "bf16", "fp16"]), bias=rng.random() < 0.5, groups=groups,
                    top_groups=top_groups, group_score=rng.choice(["max", "top2"]), renorm=rng.random() < 0.6,
                    scale=rng.choice([1.0, 2.5]), masked=rng.choice([0.0, 0.1]))
    if op == "quantize":
        return dict(op=op, rows=_spread(rng, 1, 131072), cols=8 * _spread(rng, 16, 1024),
                    dtype=rng.choice(["bf16", "fp16", "fp32"]))
    groups = rng.choice([0, 1, 8, 64, _spread(rng, 1, 64)])
    gated = rng.random() < 0.5
    return dict(op=op, rows=_spread(rng, 1, 32768), inner=16 * _spread(rng, 8, 448),
                outer=(2 if gated else 1) * _spread(rng, 32, 2048), groups=groups, gated=gated,
                dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), skew=rng.choice([0.0, 0.1, 0.5]))


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _codes(g, *shape):
    """int8 codes of normal values whose row maximum is near four deviations."""
    v = torch.randn(shape, generator=g, device=DEV, dtype=torch.float16)
    return v.mul_(32).round_().clamp_(-127, 127).to(torch.int8)


def _row_counts(case, seed):
    """Rows of each expert: a draw over skewed popularities, so that some experts stay empty."""
    r = np.random.default_rng([seed, 7])
    p = 1.0 / (1.0 + r.permutation(case["groups"])) ** case["skew"]
    return r.multinomial(case["rows"], p / p.sum())


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    if op in ("route", "route_backward"):
        T, E, K = case["T"], case["E"], case["K"]
        s["logits"] = (_randn(g, T, E) * 1.5).to(TYPES[case["dtype"]])
        width = 0.05 if case["score"] == "sigmoid" else 0.2 / E
        s["bias"] = _randn(g, E) * width if case["bias"] else None
        s["mask"] = torch.rand(T, generator=g, device=DEV) >= case["masked"] if case["masked"] else None
        if op == "route_backward":
            idx = torch.topk(s["logits"].float(), K, dim=1).indices
            if s["mask"] is not None:
                idx = torch.where(s["mask"][:, None], idx, -1)
            s["idx"] = idx
            s["grad"] = _randn(g, T, K)
    elif op == "quantize":
        # rows of different sizes, a few channels far above the rest, as activations have them
        x = _randn(g, case["rows"], case["cols"]) * torch.exp(_randn(g, case["rows"], 1))
        x[:, :: 61] *= 6
        s["x"] = x.to(TYPES[case["dtype"]])
    else:
        G, inner, outer = case["groups"], case["inner"], case["outer"]
        rows = case["rows"] + G * (ALIGN - 1)  # room for every expert's padding
        s["a"] = _codes(g, rows, inner)
        s["a_scale"] = (torch.rand(rows, generator=g, device=DEV) + 0.5) * (4 / 127)
        s["w"] = _codes(g, *((G, outer, inner) if G else (outer, inner)))
        s["w_scale"] = (torch.rand(s["w"].shape[:-1], generator=g, device=DEV) + 0.5) * (4 / 127 / math.sqrt(inner))
        width = outer // 2 if case["gated"] else outer
        s["out"] = torch.zeros((rows, width), dtype=TYPES[case["dtype"]], device=DEV)
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
    return {"route": _plain_route, "route_backward": _plain_route_backward, "quantize": _plain_quantize,
            "product": _plain_product}[c["op"]](c, state)


@functools.lru_cache(maxsize=None)
def _router(E, K, score, groups, top_groups, group_score, renorm, scale):
    import combine_topk_idx_expert_amd as ep

    return ep.RouteConfig(E=E, K=K, score=score, num_groups=groups, topk_groups=top_groups, group_score=group_score,
                          renormalize=renorm, scale=scale)


def _call(c, s):
    import combine_topk_idx_expert_amd as ep

    if c["op"] in ("route", "route_backward"):
        rc = _router(c["E"], c["K"], c["score"], c["groups"], c["top_groups"], c["group_score"], c["renorm"],
                     c["scale"])
        if c["op"] == "route":
            return ep.route(rc, s["logits"], bias=s["bias"], token_mask=s["mask"])
        return ep.route_backward(rc, s["logits"], s["idx"], s["grad"])
    if c["op"] == "quantize":
        return ep.quantize_int8(s["x"])
    rows = (s["start"], s["count"]) if c["groups"] else None
    return ep.matmul_int8((s["a"], s["a_scale"]), (s["w"], s["w_scale"]), rows=rows, gated=c["gated"], out=s["out"])


def _plain_route(c, s):
    x, E, K, G = s["logits"], c["E"], c["K"], c["groups"]
    T = x.shape[0]
    # The order of the choices is that of the exact scores; scores that differ by less than fp32 resolves are
    # common among 256 of them, so the order is taken in 64 bits.  Without a bias and without sums of scores
    # the logits themselves have that order.
    by_logit = s["bias"] is None and (G == 1 or c["group_score"] == "max")
    if by_logit:
        key = x.float()
    else:
        x64 = x.double()
        key = torch.sigmoid(x64) if c["score"] == "sigmoid" else torch.softmax(x64, 1)
        if s["bias"] is not None:
            key = key + s["bias"].double()
    if G > 1:
        per = key.view(T, G, E // G)
        if c["group_score"] == "max" or E == G:
            gs = per.amax(2)
        else:
            gs = per.topk(2, dim=2).values.sum(2)
        best = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, : c["top_groups"]]
        keep = torch.zeros((T, G), dtype=torch.bool, device=x.device).scatter_(1, best, True)
        key = torch.where(keep[:, :, None], per, -math.inf).reshape(T, E)
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :K]
    xf = x.float()
    if c["score"] == "sigmoid":
        w = torch.sigmoid(torch.gather(xf, 1, idx))
    else:
        w = torch.gather(torch.softmax(xf, 1), 1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = w * c["scale"]
    if s["mask"] is not None:
        idx = torch.where(s["mask"][:, None], idx, -1)
        w = torch.where(s["mask"][:, None], w, 0.0)
    return idx, w


def _plain_route_backward(c, s):
    x, idx, g = s["logits"].float(), s["idx"], s["grad"]
    valid = idx >= 0
    at = idx.clamp(min=0)
    g = torch.where(valid, g, 0.0)
    if c["score"] == "sigmoid":
        p = torch.sigmoid(torch.gather(x, 1, at)) * valid
    else:
        full = torch.softmax(x, 1)
        p = torch.gather(full, 1, at) * valid
    if c["renorm"]:
        total = p.sum(1, keepdim=True).clamp(min=1e-38)
        d = (g - (g * p / total).sum(1, keepdim=True)) / total
    else:
        d = g
    d = d * c["scale"]
    if c["score"] == "sigmoid":
        grad = torch.zeros_like(x).scatter_add_(1, at, d * p * (1 - p))
    else:
        inner = (d * p).sum(1, keepdim=True)
        if c["renorm"]:  # the sum is zero: nothing reaches the experts that were not chosen
            grad = torch.zeros_like(x).scatter_add_(1, at, d * p - inner * p)
        else:
            grad = (-inner * full).scatter_add_(1, at, d * p)
    return grad.to(s["logits"].dtype)


def _plain_quantize(c, s):
    # The codes are whole numbers and are held to equality, beside the scale of each row.  The quotient is taken
    # in 64 bits, where none rounds onto the border between two codes.
    x = s["x"].double()
    scale = (x.abs().amax(1, keepdim=True) / 127).float()
    q = torch.where(scale > 0, torch.round(x / scale.double()), 0.0)
    return q.clamp(-127, 127).to(torch.int8), scale[:, 0]


def _plain_product(c, s):
    a, w, out = s["a"], s["w"], s["out"]
    if c["groups"]:
        # rows of one expert side by side, as many as the fullest has
        at = s["start"][:, None] + torch.arange(max(s["most"], 1), device=a.device)
        there = torch.arange(max(s["most"], 1), device=a.device) < s["count"][:, None]
        at = torch.where(there, at, 0)
        x = a[at].float().transpose(1, 2).contiguous()
        y = torch.bmm(w.float(), x).transpose(1, 2)  # [G, most, outer]
        y = y * s["a_scale"][at][:, :, None] * s["w_scale"][:, None, :]
    else:
        y = (a.float() @ w.float().t()) * s["a_scale"][:, None] * s["w_scale"][None, :]
    if c["gated"]:
        gate, up = y.chunk(2, dim=-1)
        y = gate * torch.sigmoid(gate) * up
    y = y.to(out.dtype)
    if c["groups"]:
        out[at[there]] = y[there]
        return out
    return y


# ------------------------------------------------------------------------------------------
# what a pass cannot do without, and the values in 64 bits
# ------------------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "route":
        T, E, K = case["T"], case["E"], case["K"]
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": T * E * size + T * K * 12 + (E * 4 if case["bias"] else 0), "flops": T * E * 4}
    if op == "route_backward":
        T, E, K = case["T"], case["E"], case["K"]
        size = 4 if case["dtype"] == "fp32" else 2
        # chosen logits alone, unless the softmax runs over the whole row
        read = E if case["score"] == "softmax" and not case["renorm"] else K
        return {"bytes": T * (E + read) * size + T * K * 12, "flops": T * E}
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * ((4 if case["dtype"] == "fp32" else 2) + 1) + case["rows"] * 4, "flops": n * 4}
    G, M, inner, outer = case["groups"], case["rows"], case["inner"], case["outer"]
    width = outer // 2 if case["gated"] else outer
    experts = min(G, M) if G else 1
    return {"bytes": M * inner + experts * outer * (inner + 4) + M * 4
            + M * width * (4 if case["dtype"] == "fp32" else 2),
            "flops": 2 * M * inner * outer}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(case, s)
    if op == "route_backward":
        x = s["logits"].double().requires_grad_()
        chosen = s["idx"] >= 0
        lowest = torch.full((), -math.inf, dtype=torch.float64, device=x.device)
        # log scores, so that the renormalised weights are a softmax of them
        score = torch.nn.functional.logsigmoid(x) if case["score"] == "sigmoid" else torch.log_softmax(x, 1)
        score = torch.gather(score, 1, s["idx"].clamp(min=0))
        if case["renorm"]:
            score = score - torch.logsumexp(torch.where(chosen, score, lowest.clamp(min=-1e300)), 1, keepdim=True)
        w = torch.where(chosen, score.exp() * case["scale"], 0.0)
        (w * s["grad"].double()).sum().backward()
        return torch.nan_to_num(x.grad)
    if op == "quantize":
        x = s["x"].double()
        scale = x.abs().amax(1) / 127
        return None, scale
    a, w = s["a"].double() * s["a_scale"].double()[:, None], s["w"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    starts = s["start"].tolist() if case["groups"] else [0]
    counts = s["count"].tolist() if case["groups"] else [case["rows"]]
    for e, (lo, n) in enumerate(zip(starts, counts)):
        if n == 0:
            continue
        we = w[e] if case["groups"] else w
        ws = s["w_scale"][e] if case["groups"] else s["w_scale"]
        y = torch.nn.functional.linear(a[lo:lo + n], we.double() * ws.double()[:, None])
        if case["gated"]:
            half = y.shape[1] // 2
            y = y[:, :half] / (1 + torch.exp(-y[:, :half])) * y[:, half:]
        out[lo:lo + n] = y
    return out


def _exact_route(c, s):
    x = s["logits"].double()
    T, E = x.shape
    if c["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-x))
    else:
        score = torch.exp(x - x.amax(1, keepdim=True))
        score = score / score.sum(1, keepdim=True)
    left = score if s["bias"] is None else score + s["bias"].double()
    per = E // c["groups"]
    at = torch.arange(E, device=x.device)
    if c["groups"] > 1:
        first = left.view(T, c["groups"], per)
        gs = torch.sort(first, dim=2, descending=True).values[:, :, : 2 if c["group_score"] == "top2" else 1].sum(2)
        for _ in range(c["top_groups"]):
            best = torch.where(gs == gs.amax(1, keepdim=True), torch.arange(c["groups"], device=x.device), E).amin(1)
            gs.scatter_(1, best[:, None], -math.inf)
        left = torch.where((gs == -math.inf).repeat_interleave(per, 1), left, -math.inf)
    left = left.clone()
    chosen = []
    for _ in range(c["K"]):
        best = torch.where(left == left.amax(1, keepdim=True), at, E).amin(1)
        left.scatter_(1, best[:, None], -math.inf)
        chosen.append(best)
    idx = torch.stack(chosen, 1)
    w = torch.gather(score, 1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = w * c["scale"]
    if s["mask"] is not None:
        idx = torch.where(s["mask"][:, None], idx, -1)
        w = torch.where(s["mask"][:, None], w, 0.0)
    return idx, w

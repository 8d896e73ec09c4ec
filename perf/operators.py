"""The operators around the feed-forward layer in a language model's training step, as measurable cases.

Four operators, reached through the package's public functions:

  layernorm_fwd   y = LN(x + res) * w + b, with the sum, the means and the reciprocal deviations a backward reads
  layernorm_bwd   dx (+ the residual's gradient), dw and db of it
  xent            softmax cross entropy of a linear head x W^T over the vocabulary: losses, and with grad also dx and dW
  clip            the L2 norm over many gradient tensors, and the gradients scaled so that it is at most max_norm

A case is a dict of plain values. `prepare` makes the inputs on the GPU from a seed, `run` is one pass, `work` the bytes
and operations it cannot do without, `exact` the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

IGNORE = -100
UNSCORED = 0.06  # share of positions without a target
EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one generated token's hidden row before the feed-forward layer: latency only
        {"name": "ln_fwd_one_token", "op": "layernorm_fwd", "rows": 1, "d": 4096, "x": "bf16", "y": "bf16", "w": "f32",
         "res": False},
        # a prompt's rows at the inference layer's size, residual stream kept in 32 bits
        {"name": "ln_fwd_prompt_f32", "op": "layernorm_fwd", "rows": 4096, "d": 2048, "x": "f32", "y": "bf16", "w": "f32",
         "res": True},
        # the training step's rows, bf16 residual stream
        {"name": "ln_fwd_train", "op": "layernorm_fwd", "rows": 16384, "d": 4096, "x": "bf16", "y": "bf16", "w": "bf16",
         "res": True},
        # a ragged micro-batch of a small model in 32 bits: odd width, so no aligned rows
        {"name": "ln_bwd_ragged_f32", "op": "layernorm_bwd", "rows": 777, "d": 1001, "x": "f32", "y": "f32", "w": "f32",
         "res": False},
        # the training step's backward, with the residual branch's gradient added
        {"name": "ln_bwd_train", "op": "layernorm_bwd", "rows": 16384, "d": 4096, "x": "bf16", "y": "bf16", "w": "f32",
         "res": True},
        # scoring one short text: few rows against a whole vocabulary of odd size
        {"name": "xent_short_text", "op": "xent", "grad": False, "rows": 61, "d": 512, "vocab": 50001},
        # held-out loss at the inference layer's size
        {"name": "xent_evaluation", "op": "xent", "grad": False, "rows": 4096, "d": 2048, "vocab": 32768},
        # a ragged micro-batch of a small model: nothing is a multiple of a tile
        {"name": "xent_grad_ragged", "op": "xent", "grad": True, "rows": 777, "d": 1000, "vocab": 50001},
        # a training micro-batch at the training layer's width
        {"name": "xent_grad_train", "op": "xent", "grad": True, "rows": 8192, "d": 4096, "vocab": 65536},
        # the one-layer training demo's three gradients (W_up, b, W_down), over the bound
        {"name": "clip_one_layer", "op": "clip", "kind": "layers", "layers": 1, "d": 1024, "f": 4096, "vocab": 0,
         "tensors": 0, "total": 0, "over": True},
        # many small tensors of odd sizes (norms, biases, adapters), both types, under the bound
        {"name": "clip_many_small", "op": "clip", "kind": "many", "layers": 0, "d": 0, "f": 0, "vocab": 0,
         "tensors": 500, "total": 4000000, "over": False},
        # a model of three layers of the training size with its head
        {"name": "clip_model", "op": "clip", "kind": "layers", "layers": 3, "d": 4096, "f": 16384, "vocab": 65536,
         "tensors": 0, "total": 0, "over": True},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("layernorm_fwd", "layernorm_bwd", "xent", "xent", "clip"))
    if op.startswith("layernorm"):
        x = rng.choice(("bf16", "f32"))
        d = _log(rng, 24, 8192)
        if rng.random() < 0.5:
            d = max(8, d // 8 * 8)
        rows = _log(rng, 1, 16384)
        rows = max(1, min(rows, (16384 * 4096 if x == "bf16" else 8192 * 4096) // d))
        y = x if x == "bf16" else rng.choice(("bf16", "f32"))
        return {"op": op, "rows": rows, "d": d, "x": x, "y": y, "w": rng.choice(("bf16", "f32")), "res": rng.random() < 0.5}
    if op == "xent":
        d = max(8, _log(rng, 64, 4096) // 8 * 8)
        vocab = _log(rng, 200, 65536)
        rows = max(1, min(_log(rng, 1, 8192), 8192 * 4096 * 65536 // (d * vocab)))
        return {"op": op, "grad": rng.random() < 0.6, "rows": rows, "d": d, "vocab": vocab}
    if rng.random() < 0.5:
        return {"op": op, "kind": "layers", "layers": rng.randint(1, 3), "d": _log(rng, 64, 2048) // 8 * 8,
                "f": _log(rng, 256, 8192) // 8 * 8, "vocab": _log(rng, 1000, 32768), "tensors": 0, "total": 0,
                "over": rng.random() < 0.5}
    return {"op": op, "kind": "many", "layers": 0, "d": 0, "f": 0, "vocab": 0, "tensors": _log(rng, 1, 600),
            "total": _log(rng, 5000, 50000000), "over": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs --

def _shapes(case):
    """The gradient tensors of a clip case: (elements, type), 32-bit layer gradients and a bf16 head."""
    if case["kind"] == "layers":
        d, f = case["d"], case["f"]
        layer = [(f * d, "f32"), (f, "f32"), (f * d, "f32")]  # W_up, b, W_down
        if case["vocab"]:
            layer += [(d, "f32"), (d, "f32")]  # norm weight and bias
        return layer * case["layers"] + ([(case["vocab"] * d, "bf16")] if case["vocab"] else [])
    n = case["tensors"]
    weights = [math.exp(4.0 * math.sin(12.9898 * (i + 1))) for i in range(n)]  # sizes over a factor of 3000
    scale = case["total"] / sum(weights)
    return [(max(1, int(w * scale)), "bf16" if i % 3 == 1 else "f32") for i, w in enumerate(weights)]


def _padded(n):
    return (n + 63) // 64 * 64


def _slices(flat, shapes):
    at, out = dict.fromkeys(flat, 0), []
    for n, t in shapes:
        out.append(flat[t][at[t]:at[t] + n])
        at[t] += _padded(n)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    s = {"case": case, "op": case["op"]}
    if case["op"].startswith("layernorm"):
        rows, d = case["rows"], case["d"]
        tx, ty, tw = DTYPES[case["x"]], DTYPES[case["y"]], DTYPES[case["w"]]
        # hidden rows as models have them: channels of different spread, an offset, a few large channels
        spread = torch.exp(0.5 * randn(d)) * torch.where(torch.rand(d, device="cuda", generator=g) < 0.01, 12.0, 1.0)
        s["x"] = (randn(rows, d) * spread + 0.3).to(tx)
        s["res"] = (0.5 * randn(rows, d)).to(tx) if case["res"] else None
        s["w"] = (1 + 0.1 * randn(d)).to(tw)
        s["b"] = (0.1 * randn(d)).to(tw)
        s["mean"] = torch.empty(rows, device="cuda")
        s["rstd"] = torch.empty(rows, device="cuda")
        if case["op"] == "layernorm_fwd":
            s["y"] = torch.empty(rows, d, device="cuda", dtype=ty)
            s["sum"] = torch.empty_like(s["x"]) if case["res"] else None
        else:
            x = s["x"].float()
            s["dy"] = (0.01 * randn(rows, d)).to(ty)
            s["mean"] = x.mean(1)
            s["rstd"] = 1.0 / torch.sqrt(((x - s["mean"][:, None]) ** 2).mean(1) + EPS)
            s["res"] = (0.01 * randn(rows, d)).to(tx) if case["res"] else None
            s["dx"] = torch.empty_like(s["x"])
            s["dw"] = torch.empty(d, device="cuda")
            s["db"] = torch.empty(d, device="cuda")
            if own:
                import activation_sparse_transformer_tcgen05_gb300 as tw
                s["ws"] = torch.empty(tw.twell_layernorm_bwd_workspace_bytes(rows, d), dtype=torch.uint8, device="cuda")
    elif case["op"] == "xent":
        rows, d, vocab = case["rows"], case["d"], case["vocab"]
        s["W"] = (randn(vocab, d) * (1.5 / math.sqrt(d))).bfloat16()
        # frequent and rare words, some positions not scored, rows that lean towards their word as far as a model has learnt it
        u = torch.rand(rows, device="cuda", generator=g)
        target = (torch.exp(u * math.log(vocab)) - 1).long().clamp_(0, vocab - 1)
        lean = 2.5 * torch.rand(rows, 1, device="cuda", generator=g)
        s["x"] = (randn(rows, d) + lean * s["W"][target].float()).bfloat16()
        target[torch.rand(rows, device="cuda", generator=g) < UNSCORED] = IGNORE
        s["target"] = target
        s["nll"] = torch.empty(rows, device="cuda")
        s["lse"] = torch.empty(rows, device="cuda")
        s["loss"] = torch.empty(1, device="cuda")
        if case["grad"]:
            s["dx"] = torch.empty_like(s["x"])
            s["dW"] = torch.empty_like(s["W"])
        if own:
            import activation_sparse_transformer_tcgen05_gb300 as tw
            n = (tw.twell_xent_bwd_workspace_bytes(rows, d, vocab, rows, tw.DTYPE_BF16) if case["grad"]
                 else tw.twell_xent_fwd_workspace_bytes(rows, d, vocab))
            s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
            s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    else:
        shapes = _shapes(case)
        # layers' gradients differ in size; the bound is a tenth of the norm, or ten times it
        s["grads"] = [(randn(n) * (1e-3 * math.exp(math.sin(3.7 * i)))).to(DTYPES[t]) for i, (n, t) in enumerate(shapes)]
        norm = math.sqrt(sum(n * (1e-3 * math.exp(math.sin(3.7 * i))) ** 2 for i, (n, _) in enumerate(shapes)))
        s["max_norm"] = 0.1 * norm if case["over"] else 10.0 * norm
        # the scaled gradients go to slices of one flat buffer for each type, each slice on a 64-element boundary
        s["flat"] = {k: torch.zeros(sum(_padded(n) for n, t in shapes if t == k), device="cuda", dtype=DTYPES[k])
                     for k in DTYPES if any(t == k for _, t in shapes)}
        s["out"] = _slices(s["flat"], shapes)
        s["norm"] = torch.empty(1, device="cuda")
        if own:
            import activation_sparse_transformer_tcgen05_gb300 as tw
            s["list"] = tw.TwellTensorList(s["grads"], s["out"])
            s["ws"] = torch.empty(tw.twell_grad_clip_workspace_bytes(), dtype=torch.uint8, device="cuda")
    return s


# -------------------------------------------------------------- plain forms --

def _plain_layernorm_fwd(s):
    total = s["x"] if s["res"] is None else (s["x"].float() + s["res"].float()).to(s["x"].dtype)
    x = total.float()
    mean = x.mean(1, keepdim=True)
    centred = x - mean
    rstd = 1.0 / torch.sqrt((centred * centred).mean(1, keepdim=True) + EPS)
    y = (centred * rstd * s["w"].float() + s["b"].float()).to(s["y"].dtype)
    return [y, mean[:, 0], rstd[:, 0]] + ([] if s["res"] is None else [total])


def _plain_layernorm_bwd(s):
    dy = s["dy"].float()
    hat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    wdy = dy * s["w"].float()
    dx = s["rstd"][:, None] * (wdy - wdy.mean(1, keepdim=True) - hat * (wdy * hat).mean(1, keepdim=True))
    if s["res"] is not None:
        dx = dx + s["res"].float()
    return [dx.to(s["x"].dtype), (dy * hat).sum(0), dy.sum(0)]


def _plain_xent(s):
    x, W, target = s["x"].float(), s["W"].float(), s["target"]
    z = x @ W.t()
    counted = target != IGNORE
    at = torch.where(counted, target, 0)[:, None]
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    lse = torch.where(counted, (top + torch.log(total))[:, 0], 0.0)
    nll = torch.where(counted, lse - z.gather(1, at)[:, 0], 0.0)
    n = counted.sum().clamp(min=1).float()
    loss = (nll.sum() / n)[None]
    if not s["case"]["grad"]:
        return [nll, lse, loss]
    scale = torch.where(counted, 1.0 / n, 0.0)[:, None]
    dz = e / total * scale
    dz.scatter_add_(1, at, -scale)
    return [nll, lse, loss, (dz @ W).to(s["x"].dtype), (dz.t() @ x).to(s["W"].dtype)]


def _plain_clip(s):
    squares = torch.stack([(t.float() * t.float()).sum() for t in s["grads"]])
    norm = torch.sqrt(squares.sum())
    scale = torch.clamp(s["max_norm"] / norm, max=1.0)
    return {"norm": norm[None], **_flat(s["grads"], [(t.float() * scale).to(t.dtype) for t in s["grads"]])}


def _flat(grads, values):
    """The values joined by their gradient's type, each padded with zeros to a 64-element boundary."""
    pieces = [(g.dtype, torch.nn.functional.pad(v, (0, _padded(v.numel()) - v.numel()))) for g, v in zip(grads, values)]
    return {k: torch.cat([v for t, v in pieces if t == kind]) for k, kind in DTYPES.items()
            if any(t == kind for t, _ in pieces)}


# --------------------------------------------------------------------- run --

def run(s):
    op = s["op"]
    if not own:
        return {"layernorm_fwd": _plain_layernorm_fwd, "layernorm_bwd": _plain_layernorm_bwd, "xent": _plain_xent,
                "clip": _plain_clip}[op](s)
    import activation_sparse_transformer_tcgen05_gb300 as tw
    if op == "layernorm_fwd":
        tw.twell_layernorm_fwd(s["x"], s["res"], s["w"], s["b"], EPS, s["sum"], s["y"], s["mean"], s["rstd"])
        return [s["y"], s["mean"], s["rstd"]] + ([] if s["res"] is None else [s["sum"]])
    if op == "layernorm_bwd":
        tw.twell_layernorm_bwd(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], s["res"], s["dx"], s["dw"], s["db"], s["ws"])
        return [s["dx"], s["dw"], s["db"]]
    if op == "xent":
        if not s["case"]["grad"]:
            tw.twell_xent_fwd(s["x"], s["W"], s["target"], IGNORE, True, s["nll"], s["lse"], s["loss"], s["ws"],
                              s["status"])
            return [s["nll"], s["lse"], s["loss"]]
        tw.twell_xent_fwd_bwd(s["x"], s["W"], s["target"], IGNORE, True, 1.0, s["case"]["rows"], s["nll"], s["lse"],
                              s["loss"], s["dx"], s["dW"], False, s["ws"], s["status"])
        return [s["nll"], s["lse"], s["loss"], s["dx"], s["dW"]]
    tw.twell_grad_clip(s["list"], s["max_norm"], s["norm"], s["ws"])
    return {"norm": s["norm"], **s["flat"]}


# -------------------------------------------------------------------- work --

def work(case):
    if case["op"].startswith("layernorm"):
        n, d = case["rows"], case["d"]
        size = {"bf16": 2, "f32": 4}
        sx, sy, sw = size[case["x"]], size[case["y"]], size[case["w"]]
        if case["op"] == "layernorm_fwd":
            return {"bytes": n * d * (sx + sy + (2 * sx if case["res"] else 0)) + 2 * d * sw + 8 * n, "flops": 8 * n * d}
        return {"bytes": n * d * (2 * sx + sy + (sx if case["res"] else 0)) + d * (sw + 8) + 8 * n, "flops": 14 * n * d}
    if case["op"] == "xent":
        n, d, v = case["rows"], case["d"], case["vocab"]
        scored = (1 - UNSCORED) * n
        read = 2 * scored * d + 2 * v * d + 8 * n
        if not case["grad"]:
            return {"bytes": read + 8 * n, "flops": 2 * scored * v * d}
        # logits, dx and dW: one product each
        return {"bytes": read + 8 * n + 2 * n * d + 2 * v * d, "flops": 6 * scored * v * d}
    shapes = _shapes(case)
    each = sum(n * (2 if t == "bf16" else 4) for n, t in shapes)
    # read for the norm, then read and written scaled; what the second read finds in the cache is not taken off
    return {"bytes": 3 * each, "flops": 3 * sum(n for n, _ in shapes)}


# ------------------------------------------------------------------- exact --

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "layernorm_fwd":
        total = s["x"] if s["res"] is None else (s["x"].double() + s["res"].double()).to(s["x"].dtype)
        var, mean = torch.var_mean(total.double(), dim=1, correction=0)
        rstd = (var + EPS) ** -0.5
        y = (total.double() * rstd[:, None] - (mean * rstd)[:, None]) * s["w"].double() + s["b"].double()
        return [y, mean, rstd] + ([] if s["res"] is None else [total.double()])
    if case["op"] == "layernorm_bwd":
        # the normalised row's Jacobian: rstd (I - 11'/d - hat hat'/d), applied to w dy
        x, dy, rstd = s["x"].double(), s["dy"].double(), s["rstd"].double()[:, None]
        hat = x.sub(s["mean"].double()[:, None]).mul(rstd)
        v = dy * s["w"].double()
        d = x.shape[1]
        dx = rstd * v - rstd * (v.sum(1, keepdim=True) / d) - rstd * hat * ((v * hat).sum(1, keepdim=True) / d)
        if s["res"] is not None:
            dx += s["res"].double()
        return [dx, torch.einsum("nd,nd->d", dy, hat), torch.einsum("nd->d", dy)]
    if case["op"] == "xent":
        x, W, target = s["x"].double(), s["W"].double(), s["target"]
        z = torch.mm(x, W.T)
        rows = torch.nonzero(target != IGNORE)[:, 0]
        lse = torch.zeros(len(target), dtype=torch.float64, device="cuda")
        lse[rows] = torch.logsumexp(z[rows], dim=1)
        nll = torch.zeros_like(lse)
        nll[rows] = lse[rows] - z[rows, target[rows]]
        n = max(1, len(rows))
        if not case["grad"]:
            return [nll, lse, nll.sum()[None] / n]
        dz = torch.zeros_like(z)
        dz[rows] = torch.exp(z[rows] - lse[rows, None])
        del z
        dz[rows, target[rows]] -= 1.0
        dz /= n
        return [nll, lse, nll.sum()[None] / n, torch.mm(dz, W), torch.mm(dz.T, x)]
    norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(t.double())) ** 2 for t in s["grads"]))
    factor = s["max_norm"] / norm if norm > s["max_norm"] else 1.0
    return {"norm": torch.tensor([norm], dtype=torch.float64, device="cuda"),
            **_flat(s["grads"], [t.double() * factor for t in s["grads"]])}

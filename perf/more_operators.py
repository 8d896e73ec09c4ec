"""The gated feed-forward layer trained and served densely, linear layers, and the optimiser's step, as measurable cases.

Three operators, each with its backward pass or its state, reached through the package's public functions:

  gated_fwd    h = act(x W_gate^T + b) * (x W_up^T), y = h W_down (+ res); for training also the two pre-activations
  gated_bwd    dx, dW_gate, dW_up, dW_down and db of it, with an L1 term on h
  linear_fwd   y = act(x W^T + bias) (+ res), the logits of a head among them; for training also the pre-activation
  linear_bwd   dx, dW and dbias of it
  adamw        one step over many tensors, gradients scaled by the clipping factor, states of 32 or of 8 bits

A case is a dict of plain values. `prepare` makes the inputs on the GPU from a seed, `run` is one pass, `work` the bytes
and operations it cannot do without, `exact` the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BETA1, BETA2, ADAM_EPS, DECAY = 0.9, 0.95, 1e-8, 0.1
BLOCK = 256  # elements that share a scale of the 8-bit states
SEED = 1234  # of the optimiser's rounding
GAMMA = 0x9E3779B97F4A7C15 - (1 << 64)  # splitmix64 (Steele, Lea and Flood, 2014) in signed 64 bits
MIX1, MIX2 = 0xBF58476D1CE4E5B9 - (1 << 64), 0x94D049BB133111EB - (1 << 64)


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one generated token through the gated layer of the decode sizes: all three weights are read
        {"name": "gated_decode_1", "op": "gated_fwd", "M": 1, "d": 4096, "F": 14336, "act": "relu", "save": False, "res": True},
        # a batch of 64 sequences, one token each
        {"name": "gated_decode_64", "op": "gated_fwd", "M": 64, "d": 4096, "F": 14336, "act": "silu", "save": False,
         "res": True},
        # a prompt at the inference layer's size
        {"name": "gated_prompt", "op": "gated_fwd", "M": 4096, "d": 2048, "F": 8192, "act": "silu", "save": False, "res": True},
        # a training micro-batch, pre-activations kept for the backward
        {"name": "gated_fwd_train", "op": "gated_fwd", "M": 8192, "d": 4096, "F": 14336, "act": "relu", "save": True,
         "res": False},
        # a ragged micro-batch of a small model: nothing is a multiple of a tile
        {"name": "gated_bwd_ragged", "op": "gated_bwd", "M": 777, "d": 1000, "F": 2696, "act": "gelu", "l1": 0.0},
        # the training micro-batch's backward, L1 on the hidden activations
        {"name": "gated_bwd_train", "op": "gated_bwd", "M": 8192, "d": 4096, "F": 14336, "act": "relu", "l1": 1e-4},
        # one token's projection back into the residual stream
        {"name": "linear_one_token", "op": "linear_fwd", "M": 1, "N": 4096, "K": 4096, "act": "none", "y": "bf16", "bias": True,
         "res": True, "save": False, "kn": False},
        # logits of a few generated tokens over a vocabulary of odd size, in 32 bits
        {"name": "linear_logits", "op": "linear_fwd", "M": 61, "N": 50001, "K": 2048, "act": "none", "y": "f32", "bias": False,
         "res": False, "save": False, "kn": False},
        # a training micro-batch through a widening layer, pre-activation kept
        {"name": "linear_fwd_train", "op": "linear_fwd", "M": 8192, "N": 16384, "K": 4096, "act": "gelu_tanh", "y": "bf16",
         "bias": True, "res": False, "save": True, "kn": False},
        # its backward
        {"name": "linear_bwd_train", "op": "linear_bwd", "M": 8192, "N": 16384, "K": 4096, "act": "gelu_tanh", "bias": True,
         "kn": False},
        # many small tensors of odd sizes (norms, biases, adapters), 32-bit states, under the clipping bound
        {"name": "adamw_many_small", "op": "adamw", "kind": "many", "tensors": 500, "total": 4000000, "layers": 0, "d": 0,
         "F": 0, "vocab": 0, "p": "f32", "g": "f32", "bits": 32, "copy": True, "over": False},
        # a model of three layers of the training size with its head, 8-bit states, gradients over the clipping bound
        {"name": "adamw_model_8bit", "op": "adamw", "kind": "layers", "tensors": 0, "total": 0, "layers": 3, "d": 4096,
         "F": 16384, "vocab": 65536, "p": "f32", "g": "f32", "bits": 8, "copy": True, "over": True},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _log8(rng, low, high):
    return max(8, _log(rng, low, high) // 8 * 8)


def draw(rng):
    op = rng.choice(("gated_fwd", "gated_fwd", "gated_bwd", "linear_fwd", "linear_fwd", "linear_bwd", "adamw", "adamw"))
    act = rng.choice(("relu", "silu", "gelu", "gelu_tanh"))
    most = 8192 * 4096 * 14336
    if op.startswith("gated"):
        d, F = _log8(rng, 64, 4096), _log8(rng, 64, 14336)
        M = max(1, min(_log(rng, 1 if op == "gated_fwd" else 16, 8192), most // (d * F)))
        if op == "gated_fwd":
            return {"op": op, "M": M, "d": d, "F": F, "act": act, "save": rng.random() < 0.5, "res": rng.random() < 0.5}
        return {"op": op, "M": M, "d": d, "F": F, "act": act, "l1": rng.choice((0.0, 1e-4))}
    if op.startswith("linear"):
        act = rng.choice(("none", "none", act))
        K, N, kn = _log8(rng, 64, 4096), _log(rng, 8, 50000), rng.random() < 0.3
        if kn or rng.random() < 0.5:
            N = max(8, N // 8 * 8)
        M = max(1, min(_log(rng, 1 if op == "linear_fwd" else 16, 8192), most // (N * K)))
        if op == "linear_fwd":
            return {"op": op, "M": M, "N": N, "K": K, "act": act, "y": rng.choice(("bf16", "bf16", "f32")),
                    "bias": rng.random() < 0.6, "res": rng.random() < 0.4, "save": act != "none" and rng.random() < 0.5,
                    "kn": kn}
        return {"op": op, "M": M, "N": N, "K": K, "act": act, "bias": rng.random() < 0.6, "kn": kn}
    p, bits = rng.choice(("f32", "f32", "bf16")), rng.choice((32, 8))
    case = {"op": op, "p": p, "g": rng.choice(("f32", "bf16")), "bits": bits, "copy": p == "f32" and rng.random() < 0.6,
            "over": rng.random() < 0.5, "tensors": 0, "total": 0, "layers": 0, "d": 0, "F": 0, "vocab": 0}
    if rng.random() < 0.5:
        return {**case, "kind": "layers", "layers": rng.randint(1, 3), "d": _log8(rng, 64, 2048), "F": _log8(rng, 256, 8192),
                "vocab": _log(rng, 1000, 32768)}
    return {**case, "kind": "many", "tensors": _log(rng, 1, 600), "total": _log(rng, 5000, 50000000)}


# ------------------------------------------------------------------ inputs --

def _sizes(case):
    """Elements of an adamw case's tensors."""
    if case["kind"] == "layers":
        d, F = case["d"], case["F"]
        return [F * d, F, F * d, d, d] * case["layers"] + [case["vocab"] * d]  # W_up, b, W_down, the norm's w and b; head
    n = case["tensors"]
    weights = [math.exp(4.0 * math.sin(12.9898 * (i + 1))) for i in range(n)]  # sizes over a factor of 3000
    scale = case["total"] / sum(weights)
    return [max(1, int(w * scale)) for w in weights]


def _padded(n):
    return (n + BLOCK - 1) // BLOCK * BLOCK


def _slices(flat, sizes, per=1):
    """The tensors as slices of one flat buffer, each starting on a block's boundary (per: elements of a block's scales)."""
    at, out = 0, []
    for n in sizes:
        out.append(flat[at // per:at // per + -(-n // per)])
        at += _padded(n)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    def empty(*shape, t="bf16"):
        return torch.empty(*shape, device="cuda", dtype=DTYPES[t])

    s = {"case": case, "op": case["op"], "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if case["op"].startswith("gated"):
        M, d, F = case["M"], case["d"], case["F"]
        # hidden rows behind a norm, weights at their usual scale; a ReLU gate as sparse as an L1 term leaves it
        s["x"] = randn(M, d).bfloat16()
        s["Wg"] = (randn(F, d) * d ** -0.5).bfloat16()
        s["Wu"] = (randn(F, d) * d ** -0.5).bfloat16()
        s["Wd"] = (randn(F, d) * F ** -0.5).bfloat16()
        s["b"] = 0.2 * randn(F) - (1.3 if case["act"] == "relu" else 0.0)
        s["h"], s["y"] = empty(M, F), empty(M, d)
        if case["op"] == "gated_fwd":
            s["g"], s["u"] = (empty(M, F), empty(M, F)) if case["save"] else (None, None)
            s["res"] = randn(M, d).bfloat16() if case["res"] else None
        else:
            # what a forward has left
            gate = (s["x"].float() @ s["Wg"].float().t() + s["b"])
            up = s["x"].float() @ s["Wu"].float().t()
            s["h"] = (_act(gate, case["act"])[0] * up).bfloat16()
            s["g"], s["u"] = gate.bfloat16(), up.bfloat16()
            s["dy"] = (0.01 * randn(M, d)).bfloat16()
            s["dx"], s["dWg"], s["dWu"], s["dWd"], s["db"] = empty(M, d), empty(F, d), empty(F, d), empty(F, d), empty(F, t="f32")
            if own:
                import activation_sparse_transformer_tcgen05_gb300 as tw
                s["ws"] = empty_bytes(tw.twell_dense_gated_bwd_workspace_bytes(M, d, F))
    elif case["op"].startswith("linear"):
        M, N, K, kn = case["M"], case["N"], case["K"], case["kn"]
        s["x"] = randn(M, K).bfloat16()
        s["W"] = (randn(*((K, N) if kn else (N, K))) * K ** -0.5).bfloat16()
        s["bias"] = 0.2 * randn(N) if case["bias"] else None
        if case["op"] == "linear_fwd":
            s["res"] = randn(M, N).to(DTYPES[case["y"]]) if case["res"] else None
            s["y"] = empty(M, N, t=case["y"])
            s["pre"] = empty(M, N) if case["save"] else None
        else:
            s["pre"] = randn(M, N).bfloat16() if case["act"] != "none" else None
            s["dy"] = (0.01 * randn(M, N)).bfloat16()
            s["dx"], s["dW"] = empty(M, K), torch.empty_like(s["W"])
            s["db"] = empty(N, t="f32") if case["bias"] else None
            if own:
                import activation_sparse_transformer_tcgen05_gb300 as tw
                s["ws"] = empty_bytes(tw.twell_linear_bwd_workspace_bytes(M, N, K))
    else:
        sizes = _sizes(case)
        total = sum(_padded(n) for n in sizes)
        real = torch.zeros(total, device="cuda", dtype=torch.bool)
        for part in _slices(real, sizes):
            part.fill_(True)
        # a few steps into training: magnitudes over some powers of ten within every tensor, first moments of the gradients'
        # size, some elements that have had no gradient yet
        spread = torch.exp(1.5 * randn(total)) * 1e-3 * real
        seen = torch.rand(total, device="cuda", generator=g) < 0.95
        s["p"] = (0.02 * randn(total) * real).to(DTYPES[case["p"]])
        s["g"] = (randn(total) * spread).to(DTYPES[case["g"]])
        m = 0.3 * randn(total) * spread * seen
        v = (0.2 + torch.rand(total, device="cuda", generator=g)) * spread * spread * seen
        del spread, seen, real
        s["norm"] = torch.sqrt((s["g"].float() ** 2).sum())[None]
        s["max_norm"] = 0.1 * 1e-3 * math.sqrt(total) if case["over"] else 1e6
        s["lr"] = torch.full((1,), 1e-3, device="cuda")
        s["step"] = torch.full((1,), 7, device="cuda", dtype=torch.int32)
        s["copy"] = torch.zeros(total, device="cuda", dtype=torch.bfloat16) if case["copy"] else None
        if case["bits"] == 8:
            s["m"], s["ms"] = _encode(m, torch.zeros_like(m, dtype=torch.int32) + 32768, 4, True)
            s["v"], s["vs"] = _encode(v, torch.zeros_like(v, dtype=torch.int32) + 32768, 5, False)
            s["m_values"], s["v_values"] = (torch.zeros(total, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        else:
            s["m"], s["v"] = m, v
        s["sizes"] = sizes
        if own:
            import activation_sparse_transformer_tcgen05_gb300 as tw

            def cut(name, per=1):
                return _slices(s[name], sizes, per) if s.get(name) is not None else None

            s["list"] = tw.TwellAdamWList(cut("p"), cut("g"), cut("m"), cut("v"), cut("ms", BLOCK), cut("vs", BLOCK), cut("copy"))
            if case["bits"] == 8:
                s["out_m"], s["out_v"] = tw.TwellTensorList(cut("m_values")), tw.TwellTensorList(cut("v_values"))
    return s


def empty_bytes(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


# -------------------------------------------------------------- plain forms --

def _act(z, kind):
    """(act(z), act'(z)) in z's type."""
    if kind == "none":
        return z, torch.ones_like(z)
    if kind == "relu":
        on = z > 0
        return torch.where(on, z, 0.0), on.to(z.dtype)
    if kind == "silu":
        t = 1.0 / (1.0 + torch.exp(-z))
        return z * t, t * (1.0 + z * (1.0 - t))
    if kind == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)


def _plain_gated_fwd(s):
    x = s["x"].float()
    gate = x @ s["Wg"].float().t() + s["b"]
    up = x @ s["Wu"].float().t()
    h = (_act(gate, s["case"]["act"])[0] * up).bfloat16()
    y = h.float() @ s["Wd"].float()
    if s["res"] is not None:
        y = y + s["res"].float()
    return [h, y.bfloat16()] + ([gate.bfloat16(), up.bfloat16()] if s["case"]["save"] else [])


def _plain_gated_bwd(s):
    x, dy, gate, up, h = (s[k].float() for k in ("x", "dy", "g", "u", "h"))
    a, da = _act(gate, s["case"]["act"])
    dh = dy @ s["Wd"].float().t() + s["case"]["l1"] * torch.sign(a * up)
    dg, du = dh * up * da, dh * a
    dx = dg @ s["Wg"].float() + du @ s["Wu"].float()
    return [dx.bfloat16(), (dg.t() @ x).bfloat16(), (du.t() @ x).bfloat16(), (h.t() @ dy).bfloat16(), dg.sum(0)]


def _plain_linear_fwd(s):
    W = s["W"].float()
    pre = s["x"].float() @ (W if s["case"]["kn"] else W.t())
    if s["bias"] is not None:
        pre = pre + s["bias"]
    y = _act(pre, s["case"]["act"])[0]
    if s["res"] is not None:
        y = y + s["res"].float()
    return [y.to(s["y"].dtype)] + ([pre.bfloat16()] if s["pre"] is not None else [])


def _plain_linear_bwd(s):
    x, W, dpre, kn = s["x"].float(), s["W"].float(), s["dy"].float(), s["case"]["kn"]
    if s["pre"] is not None:
        dpre = dpre * _act(s["pre"].float(), s["case"]["act"])[1]
    dx = dpre @ (W.t() if kn else W)
    dW = x.t() @ dpre if kn else dpre.t() @ x
    return [dx.bfloat16(), dW.bfloat16()] + ([dpre.sum(0)] if s["db"] is not None else [])


# The 8-bit states: BLOCK elements share a power of two, `scale`; a code is a small float, 3 bits of fraction below 4 bits of
# exponent (first moment, with a sign) or 5 (second moment), the largest standing for 15/16 of the scale. Codes are rounded up
# or down with the probabilities that keep the mean, by 16 random bits an element; a second moment above 0 never becomes 0.
# A code is the top bits of the fp32 number that it makes next to fp32's smallest ones, so that small codes have no exponent.

def _scale(top):
    """The power of two of blocks whose largest magnitudes are `top` (fp32): the smallest one with top <= 15/16 of it."""
    bits = top.view(torch.int32)
    up = (bits >> 23) + 1 + ((bits & 0x7FFFFF) > 0x700000).int()
    return torch.where(top > 0, (up.clamp(max=254) << 23).view(torch.float32), 0.0)


def _encode(x, random, exponents, signed):
    """(codes, scales) of x in fp32 with 16 random bits an element; the last block may be short."""
    n = x.numel()
    blocks = torch.nn.functional.pad(x, (0, -n % BLOCK)).view(-1, BLOCK)
    scale = _scale(blocks.abs().amax(1))
    inv = torch.where(scale > 0, 1.0 / scale, 0.0)
    z = (blocks.abs() * inv[:, None] * 2.0 ** ((1 << exponents) - 127)).view(-1)[:n]
    code = (z.view(torch.int32) + (random << 4)) >> 20
    code = code.clamp(max=(8 << exponents) - 1)
    if signed:
        code = code | ((x.view(torch.int32) >> 24) & 128)
    else:
        code = torch.where((code == 0) & (x > 0), 1, code)
    return code.to(torch.uint8), scale


def _decode(code, scale, exponents, signed):
    """The fp32 values that codes stand for."""
    n, code = code.numel(), code.to(torch.int32)
    size = ((code & 127) if signed else code) << 20
    size = torch.nn.functional.pad(size, (0, -n % BLOCK)).view(-1, BLOCK).view(torch.float32)
    x = (size * 2.0 ** (127 - (1 << exponents)) * scale[:, None]).view(-1)[:n]
    return torch.where(code > 127, -x, x) if signed else x


def _mix(z):
    """splitmix64's output function on int64."""
    z = (z ^ ((z >> 30) & ((1 << 34) - 1))) * MIX1
    z = (z ^ ((z >> 27) & ((1 << 37) - 1))) * MIX2
    return z ^ ((z >> 31) & ((1 << 33) - 1))


def _words(step, tensor, stream, first, n, per):
    """Random 64-bit words of elements first .. first + n - 1, `per` elements to a word."""
    nth = ((2 * tensor + stream + 1) * GAMMA + (1 << 63)) % (1 << 64) - (1 << 63)
    key = _mix(_mix(step.long() * GAMMA + SEED) + nth)
    at = torch.arange(first, first + n, device="cuda") // per
    return _mix(key + (at + 1) * GAMMA)


def _random(step, tensor, n, stream):
    """16 random bits an element: (first moment's, second moment's), or those of a bf16 parameter."""
    e = torch.arange(n, device="cuda")
    if stream == 0:
        word = _words(step, tensor, 0, 0, n, 2) >> ((e & 1) * 32)
        return (word & 0xFFFF).int(), ((word >> 16) & 0xFFFF).int()
    return ((_words(step, tensor, 1, 0, n, 4) >> ((e & 3) * 16)) & 0xFFFF).int()


def _adamw_tensor(s, i, p, g, m, v, ms, vs, copy, m_values, v_values):
    """One tensor's step, in place."""
    case, step = s["case"], s["step"]
    c = torch.where(s["norm"] > s["max_norm"], s["max_norm"] / s["norm"], 1.0)
    grad = g.float() * c
    old_m, old_v = (m, v) if case["bits"] == 32 else (_decode(m, ms, 4, True), _decode(v, vs, 5, False))
    new_m = BETA1 * old_m + (1 - BETA1) * grad
    new_v = BETA2 * old_v + (1 - BETA2) * (grad * grad)
    t = step.double()
    by_m, by_v = (1 / (1 - BETA1 ** t)).float(), (1 / (1 - BETA2 ** t)).float()
    old = p.float()
    new = old - s["lr"] * (new_m * by_m / (torch.sqrt(new_v * by_v) + ADAM_EPS) + DECAY * old)
    if case["p"] == "bf16":  # up or down with the probabilities that keep the mean: most steps are smaller than half a unit
        bits = new.view(torch.int32) + _random(step, i, p.numel(), 1)
        p.copy_((bits >> 16 << 16).view(torch.float32))
    else:
        p.copy_(new)
    if copy is not None:
        copy.copy_(new)
    if case["bits"] == 32:
        m.copy_(new_m)
        v.copy_(new_v)
        return
    rm, rv = _random(step, i, p.numel(), 0)
    for new, code, scale, exponents, signed, random, values in ((new_m, m, ms, 4, True, rm, m_values),
                                                               (new_v, v, vs, 5, False, rv, v_values)):
        codes, scales = _encode(new, random, exponents, signed)
        code.copy_(codes)
        scale.copy_(scales)
        values.copy_(_decode(codes, scales, exponents, signed))


def _adamw_outputs(s):
    names = ["p", "copy"] + (["m", "v"] if s["case"]["bits"] == 32 else ["m_values", "v_values"])
    return {k: s[k] for k in names if s[k] is not None}


def _plain_adamw(s):
    sizes = s["sizes"]
    per = {"ms": BLOCK, "vs": BLOCK}
    cut = [_slices(s[k], sizes, per.get(k, 1)) if s.get(k) is not None else [None] * len(sizes)
           for k in ("p", "g", "m", "v", "ms", "vs", "copy", "m_values", "v_values")]
    [_adamw_tensor(s, i, *parts) for i, parts in enumerate(zip(*cut))]
    return _adamw_outputs(s)


# --------------------------------------------------------------------- run --

def run(s):
    op, case = s["op"], s["case"]
    if not own:
        return {"gated_fwd": _plain_gated_fwd, "gated_bwd": _plain_gated_bwd, "linear_fwd": _plain_linear_fwd,
                "linear_bwd": _plain_linear_bwd, "adamw": _plain_adamw}[op](s)
    import activation_sparse_transformer_tcgen05_gb300 as tw
    if op == "adamw":
        tw.twell_adamw(s["list"], s["lr"], s["step"], BETA1, BETA2, ADAM_EPS, DECAY, s["norm"], s["max_norm"], SEED)
        if case["bits"] == 8:
            tw.twell_adamw_values(s["list"], s["out_m"], s["out_v"])
        return _adamw_outputs(s)
    act = {"none": tw.ACT_NONE, "relu": tw.ACT_RELU, "silu": tw.ACT_SILU, "gelu": tw.ACT_GELU,
           "gelu_tanh": tw.ACT_GELU_TANH}[case["act"]]
    if op == "gated_fwd":
        tw.twell_dense_gated_ffn_fwd(s["x"], s["Wg"], s["Wu"], s["b"], s["Wd"], act, s["res"], s["g"], s["u"], s["h"], s["y"],
                                     s["status"])
        return [s["h"], s["y"]] + ([s["g"], s["u"]] if case["save"] else [])
    if op == "gated_bwd":
        tw.twell_dense_gated_ffn_bwd(s["x"], s["Wg"], s["Wu"], s["Wd"], act, s["g"], s["u"], s["h"], s["dy"], case["l1"],
                                     s["dx"], s["dWg"], s["dWu"], s["dWd"], False, s["db"], s["ws"], s["status"])
        return [s["dx"], s["dWg"], s["dWu"], s["dWd"], s["db"]]
    if op == "linear_fwd":
        tw.twell_linear_fwd(s["x"], s["W"], case["kn"], s["bias"], act, s["res"], s["pre"], s["y"], s["status"])
        return [s["y"]] + ([s["pre"]] if s["pre"] is not None else [])
    tw.twell_linear_bwd(s["dy"], s["x"], s["W"], case["kn"], act, s["pre"], s["dx"], s["dW"], False, s["db"], s["ws"],
                        s["status"])
    return [s["dx"], s["dW"]] + ([s["db"]] if s["db"] is not None else [])


# -------------------------------------------------------------------- work --

def work(case):
    if case["op"].startswith("gated"):
        M, d, F = case["M"], case["d"], case["F"]
        weights = 6 * d * F
        if case["op"] == "gated_fwd":
            rows = 2 * M * (d * (3 if case["res"] else 2) + F * (3 if case["save"] else 1))
            return {"bytes": weights + 4 * F + rows, "flops": 6 * M * d * F}
        # weights read, their gradients written; x, dy, g, u, h read, dx written
        return {"bytes": 2 * weights + 4 * F + 2 * M * (3 * d + 3 * F), "flops": 12 * M * d * F}
    if case["op"].startswith("linear"):
        M, N, K = case["M"], case["N"], case["K"]
        bias = 4 * N if case["bias"] else 0
        if case["op"] == "linear_fwd":
            y = 4 if case["y"] == "f32" else 2
            return {"bytes": 2 * N * K + bias + 2 * M * K + M * N * (y * (2 if case["res"] else 1) + (2 if case["save"] else 0)),
                    "flops": 2 * M * N * K}
        return {"bytes": 4 * N * K + bias + 4 * M * K + 2 * M * N * (1 if case["act"] == "none" else 2), "flops": 4 * M * N * K}
    n, size = sum(_sizes(case)), {"bf16": 2, "f32": 4}
    # states of 8 bits: codes read and written, with their blocks' scales, and the values they stand for written
    state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK + 4
    return {"bytes": n * (2 * size[case["p"]] + size[case["g"]] + state + (2 if case["copy"] else 0)), "flops": 16 * n}


# ------------------------------------------------------------------- exact --

def _exact_act(z, kind):
    """(act, act') from the logistic function and the normal distribution's."""
    if kind == "none":
        return z, torch.ones_like(z)
    if kind == "relu":
        return z.clamp(min=0.0), (z > 0).double()
    if kind == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * (2 * math.pi) ** -0.5 * torch.exp(z * z / -2)
    # silu and gelu_tanh: z sigmoid(a(z))
    k = (8 / math.pi) ** 0.5
    a, da = (z, 1.0) if kind == "silu" else (k * (z + 0.044715 * z ** 3), k * (1 + 0.134145 * z ** 2))
    t = torch.sigmoid(a)
    return z * t, t + z * t * torch.sigmoid(-a) * da


def _exact_codes(x, random, exponents):
    """The values (64 bits) that the 8-bit codes of x stand for."""
    n = x.numel()
    blocks = torch.nn.functional.pad(x, (0, -n % BLOCK)).view(-1, BLOCK)
    top = blocks.abs().amax(1, keepdim=True)
    frac, power = torch.frexp(top)  # top = frac 2^power, 1/2 <= frac < 1
    power = power + (frac > 15 / 16).int()
    low = 2 - (1 << exponents)  # exponent of the smallest code with a leading bit, of its scale's
    y = torch.ldexp(blocks.abs(), -power)
    step = torch.ldexp(torch.ones_like(y), (torch.frexp(y)[1] - 1).clamp(min=low - 1) - 3)
    pad = torch.nn.functional.pad(random, (0, -n % BLOCK)).view(-1, BLOCK)
    code = torch.floor(y / step + pad.double() / 65536) * step
    if exponents == 5:
        code = torch.where((code == 0) & (y > 0), step, code)
    value = torch.ldexp(torch.minimum(code, torch.full_like(code, 15 / 16)), power) * torch.sign(blocks)
    return torch.where(top > 0, value, 0.0).view(-1)[:n]


def _exact_adamw(s):
    case, sizes, per = s["case"], s["sizes"], {"ms": BLOCK, "vs": BLOCK}
    t, out = int(s["step"]), {}
    norm = float(s["norm"])
    c = s["max_norm"] / norm if norm > s["max_norm"] else 1.0
    for k, like in _adamw_outputs(s).items():
        out[k] = torch.zeros(like.numel(), dtype=torch.float64, device="cuda")
    parts = {k: _slices(s[k], sizes, per.get(k, 1)) for k in ("p", "g", "m", "v", "ms", "vs") if s.get(k) is not None}
    to = {k: _slices(v, sizes) for k, v in out.items()}
    for i, n in enumerate(sizes):
        p, g = parts["p"][i].double(), parts["g"][i].double() * c
        m, v = parts["m"][i], parts["v"][i]
        if case["bits"] == 8:
            m, v = _decode(m, parts["ms"][i], 4, True), _decode(v, parts["vs"][i], 5, False)
        m, v = torch.lerp(g, m.double(), BETA1), torch.lerp(g.square(), v.double(), BETA2)
        lr = float(s["lr"])
        p = (1 - lr * DECAY) * p - lr / (1 - BETA1 ** t) * m / (v.sqrt() / math.sqrt(1 - BETA2 ** t) + ADAM_EPS)
        if "copy" in to:
            to["copy"][i].copy_(p)
        if case["p"] == "bf16":
            unit = torch.ldexp(torch.ones_like(p), torch.frexp(p)[1].clamp(min=-125) - 8)
            p = torch.floor(p.abs() / unit + _random(s["step"], i, n, 1).double() / 65536) * unit * torch.sign(p)
        to["p"][i].copy_(p)
        if case["bits"] == 8:
            rm, rv = _random(s["step"], i, n, 0)
            to["m_values"][i].copy_(_exact_codes(m, rm, 4))
            to["v_values"][i].copy_(_exact_codes(v, rv, 5))
        else:
            to["m"][i].copy_(m)
            to["v"][i].copy_(v)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(s)
    if case["op"] == "gated_fwd":
        x = s["x"].double()
        gate = torch.addmm(s["b"].double(), x, s["Wg"].double().T)
        up = torch.mm(x, s["Wu"].double().T)
        h = up * _exact_act(gate, case["act"])[0]
        y = torch.mm(h.bfloat16().double(), s["Wd"].double())  # the layer's output is defined on h as it is kept
        if s["res"] is not None:
            y += s["res"].double()
        return [h, y] + ([gate, up] if case["save"] else [])
    if case["op"] == "gated_bwd":
        g, u, dy, x = (s[k].double() for k in ("g", "u", "dy", "x"))
        a, da = _exact_act(g, case["act"])
        dh = torch.mm(dy, s["Wd"].double().T)
        if case["l1"]:
            dh += case["l1"] * torch.sign(a) * torch.sign(u)
        du, dg = a * dh, u * da * dh
        del a, da, dh
        dx = torch.addmm(torch.mm(dg, s["Wg"].double()), du, s["Wu"].double())
        return [dx, torch.mm(dg.T, x), torch.mm(du.T, x), torch.mm(s["h"].double().T, dy), torch.einsum("mf->f", dg)]
    x, W = s["x"].double(), s["W"].double()
    if case["op"] == "linear_fwd":
        pre = torch.mm(x, W if case["kn"] else W.T)
        if s["bias"] is not None:
            pre += s["bias"].double()
        y = _exact_act(pre, case["act"])[0]
        return [y if s["res"] is None else y + s["res"].double()] + ([pre] if case["save"] else [])
    dpre = s["dy"].double()
    if case["act"] != "none":
        dpre = _exact_act(s["pre"].double(), case["act"])[1] * dpre
    dx = torch.mm(dpre, W.T if case["kn"] else W)
    dW = torch.mm(x.T, dpre) if case["kn"] else torch.mm(dpre.T, x)
    return [dx, dW] + ([torch.einsum("mn->n", dpre)] if s["db"] is not None else [])

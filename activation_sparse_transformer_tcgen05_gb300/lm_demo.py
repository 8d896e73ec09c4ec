"""Training a small language model around the activation-sparse FFN, every step through the library.

One block between an embedding and a head, on tokens of a synthetic Markov chain (each word has four successors, with
probabilities 0.7, 0.15, 0.1 and 0.05, so a model that has learnt it has a loss near the chain's entropy of 0.91 nats):

  r = E[token]                                       bf16 residual stream
  y1 = LN(r)                                         twell_layernorm_fwd
  f = relu(y1 W_up^T + b) W_down                     twell_ffn_fwd (h packed into TwELL)
  s = r + f, y2 = LN(s)                              twell_layernorm_fwd with the residual
  loss = mean cross entropy of y2 W_head^T + lam/M * sum |h|     twell_xent_fwd_bwd, l1 in twell_ffn_bwd

backward: twell_xent_fwd_bwd (dy2, dW_head), twell_layernorm_bwd, twell_ffn_bwd, twell_layernorm_bwd with the residual's
gradient; then twell_grad_clip over all gradients, and Adam on fp32 master weights: torch's operations, or twell_adamw
with states of 32 or 8 bits, which takes the norm alone from twell_grad_clip, scales the gradients as it reads them and
writes the bf16 weights of the next step. Some positions have no target. Held-out loss by twell_xent_fwd, continuations
of a text by the head's logits (twell_linear_fwd).

GatedModel trains the gated layer, f = (relu(y1 W_gate^T + b) * (y1 W_up^T)) W_down, densely (twell_dense_gated_ffn_fwd
and _bwd with the same L1 term); its held-out loss and its continuations come from the packed layer (twell_ffn_fwd with
W_gate), which visits only the units whose gate is open. Run with ``python -m
activation_sparse_transformer_tcgen05_gb300.lm_demo [--steps N] [--max-norm C] [--gated] [--optimizer adamw8]``.
"""
from __future__ import annotations

import argparse
import time

import torch

from . import twell as tw

IGNORE = -100
EPS = 1e-5
SUCCESSORS = (0.7, 0.15, 0.1, 0.05)
BETAS, ADAM_EPS = (0.9, 0.99), 1e-8
OPTIMIZERS = ("torch", "adamw", "adamw8")


class Chain:
    """Tokens whose successor is one of four fixed words."""

    def __init__(self, vocab: int, g: torch.Generator):
        self.vocab, self.g = vocab, g
        self.next = torch.randint(0, vocab, (vocab, 4), device="cuda", generator=g)
        self.p = torch.tensor(SUCCESSORS, device="cuda")

    def batch(self, n: int, unscored: float = 0.05):
        """n tokens and their targets, a share of them without one."""
        tokens = torch.randint(0, self.vocab, (n,), device="cuda", generator=self.g)
        which = torch.multinomial(self.p.expand(n, 4), 1, generator=self.g)[:, 0]
        targets = self.next[tokens, which]
        targets[torch.rand(n, device="cuda", generator=self.g) < unscored] = IGNORE
        return tokens, targets


class Model:
    """Parameters (fp32 masters), gradients and buffers of the block; forward_backward fills the gradients."""

    def __init__(self, M: int, d: int, F: int, vocab: int, T: int, g: torch.Generator):
        self.M, self.d, self.F, self.vocab, self.T = M, d, F, vocab, T

        def randn(*shape, scale):
            return torch.randn(*shape, device="cuda", generator=g) * scale

        self.params = {
            "E": randn(vocab, d, scale=1.0),
            "w1": torch.ones(d, device="cuda"), "b1": torch.zeros(d, device="cuda"),
            "W_up": randn(F, d, scale=d ** -0.5), "b": torch.zeros(F, device="cuda"), "W_down": randn(F, d, scale=F ** -0.5),
            "w2": torch.ones(d, device="cuda"), "b2": torch.zeros(d, device="cuda"),
            "W_head": randn(vocab, d, scale=0.5 * d ** -0.5),
        }
        self._extra_params(randn)
        self.grads = {k: torch.zeros_like(p) for k, p in self.params.items()}
        self.grad_list = tw.TwellTensorList(self.grads.values())
        self.copies = None  # bf16 weights that an optimiser keeps up to date

        def bf16(*shape):
            return torch.empty(*shape, device="cuda", dtype=torch.bfloat16)

        def f32(n):
            return torch.empty(n, device="cuda")

        self.y1, self.f, self.s, self.y2 = (bf16(M, d) for _ in range(4))
        self.dy2, self.ds, self.dy1, self.dr = (bf16(M, d) for _ in range(4))
        self.stats = [f32(M) for _ in range(4)]
        self.nll, self.lse, self.loss, self.norm = f32(M), f32(M), f32(1), f32(1)
        self.h = tw.TwellBuffers(M, F, T, M * F)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

        def ws(n):
            return torch.empty(n, dtype=torch.uint8, device="cuda")

        self._ffn_buffers(bf16, ws)
        self.ws_ln = ws(tw.twell_layernorm_bwd_workspace_bytes(M, d))
        self.ws_xent = ws(tw.twell_xent_bwd_workspace_bytes(M, d, vocab, 0, tw.DTYPE_F32))
        self.ws_clip = ws(tw.twell_grad_clip_workspace_bytes())

    MATRICES = ("E", "W_up", "W_down", "W_head")

    def _extra_params(self, randn):
        pass

    def _ffn_buffers(self, bf16, ws):
        M, d, F, T = self.M, self.d, self.F, self.T
        self.ws_fwd = ws(tw.twell_workspace_bytes(tw.OP_FFN_FWD, M, d, F, T, M * F))
        self.ws_bwd = ws(tw.twell_workspace_bytes(tw.OP_FFN_BWD, M, d, F, T, M * F))

    def _ffn_fwd(self, bf, training):
        tw.twell_ffn_fwd(self.y1, bf["W_up"], None, self.params["b"], bf["W_down"], self.T, self.h, self.f, self.ws_fwd,
                         self.status)

    def _ffn_bwd(self, bf, l1):
        g = self.grads
        tw.twell_ffn_bwd(self.y1, bf["W_up"], bf["W_down"], self.h, self.ds, l1, self.dy1, g["W_up"], g["W_down"], g["b"],
                         self.ws_bwd, self.status)

    def density(self):
        """Share of the last forward's hidden units that were active."""
        return float(self.h.nnz.sum()) / (self.M * self.F)

    def _weights(self):
        if self.copies is not None:
            return self.copies
        return {k: self.params[k].to(torch.bfloat16) for k in self.MATRICES}

    def _hidden(self, tokens, bf, training=False):
        """y2 of the tokens; keeps what the backward reads."""
        p, (m1, r1, m2, r2) = self.params, self.stats
        r = bf["E"][tokens]
        tw.twell_layernorm_fwd(r, None, p["w1"], p["b1"], EPS, None, self.y1, m1, r1)
        self._ffn_fwd(bf, training)
        tw.twell_layernorm_fwd(r, self.f, p["w2"], p["b2"], EPS, self.s, self.y2, m2, r2)
        return r

    def forward_backward(self, tokens, targets, lam: float):
        p, g, (m1, r1, m2, r2) = self.params, self.grads, self.stats
        bf = self._weights()
        r = self._hidden(tokens, bf, training=True)
        tw.twell_xent_fwd_bwd(self.y2, bf["W_head"], targets, IGNORE, True, 1.0, 0, self.nll, self.lse, self.loss, self.dy2,
                              g["W_head"], False, self.ws_xent, self.status)
        tw.twell_layernorm_bwd(self.dy2, self.s, p["w2"], m2, r2, None, self.ds, g["w2"], g["b2"], self.ws_ln)
        self._ffn_bwd(bf, lam / self.M)
        tw.twell_layernorm_bwd(self.dy1, r, p["w1"], m1, r1, self.ds, self.dr, g["w1"], g["b1"], self.ws_ln)
        g["E"].zero_().index_add_(0, tokens, self.dr.float())
        return self.loss

    def clip(self, max_norm: float):
        """Scales all gradients in place so that their norm is at most max_norm; the norm before is in self.norm."""
        tw.twell_grad_clip(self.grad_list, max_norm, self.norm, self.ws_clip)

    def evaluate(self, tokens, targets):
        bf = self._weights()
        self._hidden(tokens, bf)
        tw.twell_xent_fwd(self.y2, bf["W_head"], targets, IGNORE, True, self.nll, self.lse, self.loss, self.ws_xent,
                          self.status)
        return float(self.loss)

    def logits(self, tokens):
        """fp32 logits of the words that may follow each of up to M tokens."""
        n = tokens.numel()
        self._hidden(torch.nn.functional.pad(tokens, (0, self.M - n)), bf := self._weights())
        z = torch.empty(n, self.vocab, device="cuda")
        tw.twell_linear_fwd(self.y2[:n], bf["W_head"], False, None, tw.ACT_NONE, None, None, z, self.status)
        return z

    def continue_text(self, tokens, length: int):
        """The tokens followed by the likeliest word, `length` times: [n, length + 1]."""
        text = [tokens]
        for _ in range(length):
            text.append(self.logits(text[-1]).argmax(1))
        return torch.stack(text, 1)

    def check(self):
        code = tw.twell_check(self.status)
        if code != 0:
            raise RuntimeError(f"device status {code}: {tw.twell_status_string(code)}")


class GatedModel(Model):
    """The block with the gated layer, trained densely and served packed."""

    MATRICES = ("E", "W_gate", "W_up", "W_down", "W_head")

    def _extra_params(self, randn):
        self.params["W_gate"] = randn(self.F, self.d, scale=self.d ** -0.5)

    def _ffn_buffers(self, bf16, ws):
        M, d, F, T = self.M, self.d, self.F, self.T
        self.g, self.u, self.hd = (bf16(M, F) for _ in range(3))
        self.ws_fwd = ws(tw.twell_workspace_bytes(tw.OP_GATED_FWD, M, d, F, T, M * F))
        self.ws_bwd = ws(tw.twell_dense_gated_bwd_workspace_bytes(M, d, F))
        self.dense = False

    def _ffn_fwd(self, bf, training):
        b, self.dense = self.params["b"], training
        if training:
            tw.twell_dense_gated_ffn_fwd(self.y1, bf["W_gate"], bf["W_up"], b, bf["W_down"], tw.ACT_RELU, None, self.g, self.u,
                                         self.hd, self.f, self.status)
        else:
            tw.twell_ffn_fwd(self.y1, bf["W_up"], bf["W_gate"], b, bf["W_down"], self.T, self.h, self.f, self.ws_fwd,
                             self.status)

    def _ffn_bwd(self, bf, l1):
        g = self.grads
        tw.twell_dense_gated_ffn_bwd(self.y1, bf["W_gate"], bf["W_up"], bf["W_down"], tw.ACT_RELU, self.g, self.u, self.hd, self.ds,
                                     l1, self.dy1, g["W_gate"], g["W_up"], g["W_down"], False, g["b"], self.ws_bwd, self.status)

    def density(self):
        return float((self.g > 0).float().mean()) if self.dense else super().density()


class TorchAdam:
    """Clipping in place, then Adam by torch operations."""

    def __init__(self, model, lr: float, max_norm: float):
        self.model, self.lr, self.max_norm, self.t = model, lr, max_norm, 0
        self.m = {k: torch.zeros_like(p) for k, p in model.params.items()}
        self.v = {k: torch.zeros_like(p) for k, p in model.params.items()}

    def clip(self):
        self.model.clip(self.max_norm)

    def step(self):
        self.t += 1
        (b1, b2), m, v = BETAS, self.m, self.v
        for k, p in self.model.params.items():
            g = self.model.grads[k]
            m[k].lerp_(g, 1 - b1)
            v[k].mul_(b2).addcmul_(g, g, value=1 - b2)
            p.addcdiv_(m[k] / (1 - b1 ** self.t), (v[k] / (1 - b2 ** self.t)).sqrt_().add_(ADAM_EPS), value=-self.lr)


class TwellAdamW:
    """The norm by twell_grad_clip, everything else in one twell_adamw: clipping, states of 32 or 8 bits, bf16 copies.
    A norm that is not finite drops the step."""

    def __init__(self, model, lr: float, max_norm: float, bits: int = 32, weight_decay: float = 0.0, seed: int = 0):
        self.model, self.max_norm, self.weight_decay, self.seed = model, max_norm, weight_decay, seed
        params = model.params
        self.lr = torch.full((1,), lr, device="cuda")
        self.step_number = torch.zeros(1, dtype=torch.int32, device="cuda")
        model.copies = {k: params[k].to(torch.bfloat16) for k in model.MATRICES}
        kind = torch.float32 if bits == 32 else torch.uint8
        self.m, self.v = ([torch.zeros_like(p, dtype=kind) for p in params.values()] for _ in range(2))
        scales = [None, None]
        if bits == 8:
            scales = [[torch.zeros(-(-p.numel() // tw.ADAMW_BLOCK), device="cuda") for p in params.values()] for _ in range(2)]
        self.list = tw.TwellAdamWList(params.values(), model.grads.values(), self.m, self.v, *scales,
                                      copies=[model.copies.get(k) for k in params])

    def clip(self):
        self.model.clip(float("inf"))  # the norm alone

    def step(self):
        self.step_number += 1
        tw.twell_adamw(self.list, self.lr, self.step_number, *BETAS, ADAM_EPS, self.weight_decay, self.model.norm, self.max_norm,
                       self.seed)


def train(steps: int = 600, M: int = 4096, d: int = 256, F: int = 1024, vocab: int = 2000, T: int = 128, lam: float = 0.001,
          lr: float = 3e-3, max_norm: float = 1.0, seed: int = 0, log_every: int = 100, verbose: bool = True,
          gated: bool = False, optimizer: str = "torch"):
    """Runs the demo; returns the per-log history (training and held-out loss, gradient norm, hidden density, ms)."""
    if optimizer not in OPTIMIZERS:
        raise ValueError(f"optimizer must be one of {OPTIMIZERS}, got {optimizer!r}")
    g = torch.Generator(device="cuda").manual_seed(seed)
    chain = Chain(vocab, g)
    held_out = chain.batch(M)
    model = (GatedModel if gated else Model)(M, d, F, vocab, T, g)
    opt = (TorchAdam(model, lr, max_norm) if optimizer == "torch"
           else TwellAdamW(model, lr, max_norm, bits=8 if optimizer == "adamw8" else 32))
    hist = []
    if verbose:
        print(f"{'step':>6} {'loss':>8} {'held out':>9} {'norm':>8} {'density':>8} {'ms/step':>8}")
    for s in range(1, steps + 1):
        tokens, targets = chain.batch(M)
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
        model.forward_backward(tokens, targets, lam)
        opt.clip()
        e1.record()
        opt.step()
        if s == 1 or s % log_every == 0 or s == steps:
            row = {"step": s, "loss": float(model.loss), "norm": float(model.norm),
                   "density": model.density(), "ms": e0.elapsed_time(e1)}
            row["held_out"] = model.evaluate(*held_out)
            model.check()
            hist.append(row)
            if verbose:
                print(f"{s:6d} {row['loss']:8.4f} {row['held_out']:9.4f} {row['norm']:8.4f} {row['density']:8.4f} "
                      f"{row['ms']:8.3f}")
    return hist


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--steps", type=int, default=600)
    ap.add_argument("--M", type=int, default=4096)
    ap.add_argument("--d", type=int, default=256)
    ap.add_argument("--F", type=int, default=1024)
    ap.add_argument("--vocab", type=int, default=2000)
    ap.add_argument("--lam", type=float, default=0.001)
    ap.add_argument("--lr", type=float, default=3e-3)
    ap.add_argument("--max-norm", type=float, default=1.0)
    ap.add_argument("--gated", action="store_true", help="the gated layer, trained densely and evaluated packed")
    ap.add_argument("--optimizer", choices=OPTIMIZERS, default="torch")
    args = ap.parse_args(argv)
    t0 = time.time()
    train(args.steps, args.M, args.d, args.F, args.vocab, lam=args.lam, lr=args.lr, max_norm=args.max_norm,
          gated=args.gated, optimizer=args.optimizer)
    print(f"wall {time.time() - t0:.1f} s")


if __name__ == "__main__":
    main()

"""Training a small language model around the activation-sparse FFN, every step through the library.

One block between an embedding and a head, on tokens of a synthetic Markov chain (each word has four successors, with
probabilities 0.7, 0.15, 0.1 and 0.05, so a model that has learnt it has a loss near the chain's entropy of 0.91 nats):

  r = E[token]                                       bf16 residual stream
  y1 = LN(r)                                         twell_layernorm_fwd
  f = relu(y1 W_up^T + b) W_down                     twell_ffn_fwd (h packed into TwELL)
  s = r + f, y2 = LN(s)                              twell_layernorm_fwd with the residual
  loss = mean cross entropy of y2 W_head^T + lam/M * sum |h|     twell_xent_fwd_bwd, l1 in twell_ffn_bwd

backward: twell_xent_fwd_bwd (dy2, dW_head), twell_layernorm_bwd, twell_ffn_bwd, twell_layernorm_bwd with the residual's
gradient; then twell_grad_clip over all gradients, and Adam on fp32 master weights (torch; the optimiser is not part of
the library). Some positions have no target. Held-out loss by twell_xent_fwd. Run with ``python -m
activation_sparse_transformer_tcgen05_gb300.lm_demo [--steps N] [--max-norm C]``.
"""
from __future__ import annotations

import argparse
import time

import torch

from . import twell as tw

IGNORE = -100
EPS = 1e-5
SUCCESSORS = (0.7, 0.15, 0.1, 0.05)


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
        self.grads = {k: torch.zeros_like(p) for k, p in self.params.items()}
        self.grad_list = tw.TwellTensorList(self.grads.values())

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

        self.ws_fwd = ws(tw.twell_workspace_bytes(tw.OP_FFN_FWD, M, d, F, T, M * F))
        self.ws_bwd = ws(tw.twell_workspace_bytes(tw.OP_FFN_BWD, M, d, F, T, M * F))
        self.ws_ln = ws(tw.twell_layernorm_bwd_workspace_bytes(M, d))
        self.ws_xent = ws(tw.twell_xent_bwd_workspace_bytes(M, d, vocab, 0, tw.DTYPE_F32))
        self.ws_clip = ws(tw.twell_grad_clip_workspace_bytes())

    def _weights(self):
        return {k: self.params[k].to(torch.bfloat16) for k in ("E", "W_up", "W_down", "W_head")}

    def _hidden(self, tokens, bf):
        """y2 of the tokens; keeps what the backward reads."""
        p, (m1, r1, m2, r2) = self.params, self.stats
        r = bf["E"][tokens]
        tw.twell_layernorm_fwd(r, None, p["w1"], p["b1"], EPS, None, self.y1, m1, r1)
        tw.twell_ffn_fwd(self.y1, bf["W_up"], None, p["b"], bf["W_down"], self.T, self.h, self.f, self.ws_fwd, self.status)
        tw.twell_layernorm_fwd(r, self.f, p["w2"], p["b2"], EPS, self.s, self.y2, m2, r2)
        return r

    def forward_backward(self, tokens, targets, lam: float):
        p, g, (m1, r1, m2, r2) = self.params, self.grads, self.stats
        bf = self._weights()
        r = self._hidden(tokens, bf)
        tw.twell_xent_fwd_bwd(self.y2, bf["W_head"], targets, IGNORE, True, 1.0, 0, self.nll, self.lse, self.loss, self.dy2,
                              g["W_head"], False, self.ws_xent, self.status)
        tw.twell_layernorm_bwd(self.dy2, self.s, p["w2"], m2, r2, None, self.ds, g["w2"], g["b2"], self.ws_ln)
        tw.twell_ffn_bwd(self.y1, bf["W_up"], bf["W_down"], self.h, self.ds, lam / self.M, self.dy1, g["W_up"], g["W_down"],
                         g["b"], self.ws_bwd, self.status)
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

    def check(self):
        code = tw.twell_check(self.status)
        if code != 0:
            raise RuntimeError(f"device status {code}: {tw.twell_status_string(code)}")


def train(steps: int = 600, M: int = 4096, d: int = 256, F: int = 1024, vocab: int = 2000, T: int = 128, lam: float = 0.001,
          lr: float = 3e-3, max_norm: float = 1.0, seed: int = 0, log_every: int = 100, verbose: bool = True):
    """Runs the demo; returns the per-log history (training and held-out loss, gradient norm, hidden density, ms)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    chain = Chain(vocab, g)
    held_out = chain.batch(M)
    model = Model(M, d, F, vocab, T, g)
    m = {k: torch.zeros_like(p) for k, p in model.params.items()}
    v = {k: torch.zeros_like(p) for k, p in model.params.items()}
    b1, b2 = 0.9, 0.99
    hist = []
    if verbose:
        print(f"{'step':>6} {'loss':>8} {'held out':>9} {'norm':>8} {'density':>8} {'ms/step':>8}")
    for s in range(1, steps + 1):
        tokens, targets = chain.batch(M)
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
        model.forward_backward(tokens, targets, lam)
        model.clip(max_norm)
        e1.record()
        for k, p in model.params.items():
            m[k].lerp_(model.grads[k], 1 - b1)
            v[k].mul_(b2).addcmul_(model.grads[k], model.grads[k], value=1 - b2)
            p.addcdiv_(m[k] / (1 - b1 ** s), (v[k] / (1 - b2 ** s)).sqrt_().add_(1e-8), value=-lr)
        if s == 1 or s % log_every == 0 or s == steps:
            row = {"step": s, "loss": float(model.loss), "norm": float(model.norm),
                   "density": float(model.h.nnz.sum()) / (M * F), "ms": e0.elapsed_time(e1)}
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
    args = ap.parse_args(argv)
    t0 = time.time()
    train(args.steps, args.M, args.d, args.F, args.vocab, lam=args.lam, lr=args.lr, max_norm=args.max_norm)
    print(f"wall {time.time() - t0:.1f} s")


if __name__ == "__main__":
    main()

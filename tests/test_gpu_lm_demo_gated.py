"""The gated model, trained densely with twell_adamw, evaluated by the packed layer, and its logits: everything together."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from activation_sparse_transformer_tcgen05_gb300 import build as _build
    _build.build()
from activation_sparse_transformer_tcgen05_gb300 import lm_demo  # noqa: E402
import activation_sparse_transformer_tcgen05_gb300 as tw  # noqa: E402


def test_step_gradients_match_the_model_in_64_bits():
    """As for the ReLU layer's model: every gradient as a vector within 3 % of the 64-bit one (about ten roundings to bf16
    on the way, 2^-9 rms each), the embedding's and the first norm's, behind gates that may switch, within 5 %."""
    g = torch.Generator(device="cuda").manual_seed(3)
    M, d, F, vocab, lam = 384, 64, 256, 500, 0.02
    chain = lm_demo.Chain(vocab, g)
    model = lm_demo.GatedModel(M, d, F, vocab, 16, g)
    tokens, targets = chain.batch(M)
    loss = float(model.forward_backward(tokens, targets, lam))
    model.check()

    P = {k: (v.to(torch.bfloat16) if k in model.MATRICES else v).double().requires_grad_() for k, v in model.params.items()}

    def norm(x, w, b):
        c = x - x.mean(1, keepdim=True)
        return c / torch.sqrt((c * c).mean(1, keepdim=True) + lm_demo.EPS) * w + b

    r = P["E"][tokens]
    y1 = norm(r, P["w1"], P["b1"])
    h = torch.relu(y1 @ P["W_gate"].T + P["b"]) * (y1 @ P["W_up"].T)
    y2 = norm(r + h @ P["W_down"], P["w2"], P["b2"])
    keep = targets != lm_demo.IGNORE
    z = (y2 @ P["W_head"].T)[keep]
    ref = (torch.logsumexp(z, 1) - z.gather(1, targets[keep][:, None])[:, 0]).mean()
    (ref + lam / M * h.abs().sum()).backward()
    assert abs(loss - float(ref.detach())) < 2e-2 * float(ref.detach())
    for k, p in P.items():
        err = float((model.grads[k].double() - p.grad).norm() / p.grad.norm())
        assert err < (5e-2 if k in ("E", "w1", "b1") else 3e-2), (k, err)


def _setup(bits, gated=True, seed=5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    M, d, F, vocab = 256, 64, 256, 300
    chain = lm_demo.Chain(vocab, g)
    model = (lm_demo.GatedModel if gated else lm_demo.Model)(M, d, F, vocab, 16, g)
    return chain, model, lm_demo.TwellAdamW(model, 3e-3, 0.5, bits)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("bits", [32, 8])
def test_steps_follow_torch_operations(gated, bits):
    """A few whole steps: parameters after each as the same formulas in torch give them from the same gradients, the
    clipping factor and the bf16 copies included (2^-18 of the step; 8-bit states are read back by twell_adamw_values)."""
    chain, model, opt = _setup(bits, gated)
    names = list(model.params)
    for t in range(1, 4):
        tokens, targets = chain.batch(model.M)
        model.forward_backward(tokens, targets, 0.01)
        opt.clip()
        if bits == 8:
            m, v = ([torch.empty_like(p) for p in model.params.values()] for _ in range(2))
            tw.twell_adamw_values(opt.list, tw.TwellTensorList(m), tw.TwellTensorList(v))
        else:
            m, v = opt.m, opt.v
        m, v = [t_.double() for t_ in m], [t_.double() for t_ in v]
        before = {k: p.double() for k, p in model.params.items()}
        opt.step()
        model.check()
        c = min(1.0, 0.5 / float(model.norm))
        for i, k in enumerate(names):
            g = model.grads[k].double() * c
            b1, b2 = lm_demo.BETAS
            m1, v1 = b1 * m[i] + (1 - b1) * g, b2 * v[i] + (1 - b2) * g * g
            under = (v1 / (1 - b2 ** t)).sqrt() + lm_demo.ADAM_EPS
            step = 3e-3 * m1 / (1 - b1 ** t) / under
            # a first moment near 0 is as exact as its terms
            most = 3e-3 * (b1 * m[i].abs() + (1 - b1) * g.abs()) / (1 - b1 ** t) / under
            off = (model.params[k].double() - (before[k] - step)).abs()
            assert bool((off <= 2.0 ** -18 * most + 2.0 ** -23 * before[k].abs() + 1e-30).all()), k
            if k in model.copies:
                assert torch.equal(model.copies[k], model.params[k].to(torch.bfloat16))


def test_packed_evaluation_agrees_with_the_dense_forward():
    """The held-out loss by the packed layer and by the dense one: both round h and y once, so rows differ by a few
    roundings of bf16 and the mean of 256 losses by less than 2^-8 of itself."""
    chain, model, opt = _setup(32)
    tokens, targets = chain.batch(model.M)
    packed = model.evaluate(tokens, targets)
    assert model.density() < 1
    dense = float(model.forward_backward(tokens, targets, 0.0))
    assert abs(packed - dense) <= 2.0 ** -8 * dense


def test_logits_are_what_the_loss_sees():
    """Log-softmax of the logits at the targets against the losses of the cross entropy (logits within 1e-5, plus fp32)."""
    chain, model, opt = _setup(32, gated=False)
    tokens, targets = chain.batch(model.M)
    z = model.logits(tokens)
    model.evaluate(tokens, targets)
    keep = targets != lm_demo.IGNORE
    nll = torch.logsumexp(z.double(), 1) - z.double().gather(1, targets.clamp(min=0)[:, None])[:, 0]
    assert bool(((nll - model.nll.double()).abs()[keep] <= 2e-5 * (1 + z.abs().amax(1).double()[keep])).all())
    few = model.logits(tokens[:5])  # another number of rows, another kernel: sums in another order
    assert bool(((few - z[:5]).abs() <= 1e-5 * (1 + z[:5].abs())).all())
    text = model.continue_text(tokens[:3], 4)
    assert text.shape == (3, 5) and torch.equal(text[:, 0], tokens[:3])
    assert torch.equal(text[:, 1], few[:3].argmax(1))


@pytest.mark.parametrize("optimizer", ["adamw", "adamw8"])
@pytest.mark.parametrize("gated", [False, True])
def test_training_runs(gated, optimizer):
    hist = lm_demo.train(steps=5, M=512, d=64, F=128, vocab=200, T=64, log_every=5, verbose=False, gated=gated, optimizer=optimizer)
    assert [row["step"] for row in hist] == [1, 5]
    assert all(torch.isfinite(torch.tensor([row["loss"], row["held_out"], row["norm"]])).all() for row in hist)
    with pytest.raises(ValueError):
        lm_demo.train(steps=1, optimizer="sgd", verbose=False)

"""The operators together: the example language model trains, its gradients are
those of the same model written in plain float32 torch, and generating token by
token gives what the whole sequence gives."""
import importlib.util
import os

import pytest
import torch

from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "language_model.py")


@pytest.fixture(scope="module")
def lm():
    spec = importlib.util.spec_from_file_location("language_model", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def plain_loss(model, tokens, targets, resets):
    """The model in plain torch on the CPU, the projections' operands rounded to
    bf16 as the kernels' are (the gradients straight through)."""
    def rounded(x):
        return x + (x.bfloat16().float() - x).detach()
    P = {k: v.detach().double().cpu().requires_grad_(True) for k, v in model.named_parameters()}
    D, layers = model.width, len(model.w_in)

    def norm(v, w):
        return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + 1e-6) * w
    x = P["embedding"][tokens.cpu()]
    z = norm(x, P["w_pre.0"])
    keep = (~resets.cpu()).double()
    for layer in range(layers):
        u = rounded(rounded(z) @ rounded(P[f"w_in.{layer}"]).t())
        r, i, v, g = (u[..., k * D:(k + 1) * D] for k in range(4))
        log_a = -8.0 * torch.nn.functional.softplus(P[f"lam.{layer}"]) * torch.sigmoid(r)
        b = torch.sqrt(-torch.expm1(2 * log_a)) * torch.sigmoid(i) * v
        h, states = torch.zeros_like(b[:, 0]), []
        for t in range(b.shape[1]):
            h = keep[:, t, None] * torch.exp(log_a[:, t]) * h + b[:, t]
            states.append(h)
        h = torch.stack(states, 1)
        x = x + model.scale * norm(h * g * torch.sigmoid(g), P[f"w_post.{layer}"])
        z = norm(x, P[f"w_pre.{layer + 1}"])
    logits = rounded(rounded(z) @ rounded(P["head"]).t())
    logp = torch.log_softmax(logits, -1)
    t = targets.cpu()
    score = logp.gather(-1, t.clamp(min=0)[..., None])[..., 0]
    loss = -(score * (t >= 0)).sum() / (t >= 0).sum()
    loss.backward()
    return loss.item(), {k: v.grad for k, v in P.items()}


def test_gradients_are_the_plain_models(lm):
    """Gradients pass through bf16 (du, dz, dlogits: 2^-9 each, about ten such
    roundings of independent elements on a path): 2 % of each gradient's norm."""
    model = lm.LanguageModel(vocabulary=50, width=32, layers=2, device=DEV)
    tokens, targets, resets = lm.synthetic_batch(2, 70, 50, seed=3, device=DEV)
    loss = model.loss(tokens, targets, resets)
    loss.backward()
    want, grads = plain_loss(model, tokens, targets, resets)
    assert abs(float(loss.detach()) - want) <= 5e-3 * want
    for name, p in model.named_parameters():
        g, e = p.grad.double().cpu(), grads[name]
        assert float((g - e).norm()) <= 0.02 * float(e.norm()), name


def test_it_learns(lm):
    model = lm.LanguageModel(vocabulary=64, width=128, layers=2, device=DEV)
    losses = lm.train(model, 30, batch=4, length=192, vocabulary=64)
    assert sum(losses[-5:]) / 5 < 0.6 * losses[0]


def test_generating_follows_the_whole_sequence(lm):
    """The head's input after each step is that of the whole sequence: bf16
    roundings of the stream's norm, and of the projections between the layers."""
    model = lm.LanguageModel(vocabulary=40, width=64, layers=2, device=DEV, seed=1)
    tokens = torch.randint(0, 40, (3, 24), device=DEV)
    with torch.no_grad():
        whole = model.hidden(tokens).float()
    pools = [torch.zeros((5, 64), device=DEV) for _ in model.w_in]
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device=DEV)
    for b, slot in enumerate(slots.tolist()):
        z = model.prefill(pools, slot, tokens[b, :12])
        assert float((z.float() - whole[b, 11]).abs().max()) <= 0.05
    for t in range(12, 24):
        z = model.step(pools, slots, tokens[:, t].contiguous()).float()
        assert float((z - whole[:, t]).abs().max()) <= 0.05, t


def test_generate(lm):
    model = lm.LanguageModel(vocabulary=40, width=64, layers=1, device=DEV)
    prompts = [torch.arange(n, device=DEV) % 40 for n in (1, 7, 30)]
    tokens, logprobs, entropies = model.generate(prompts, 6, top=3)
    again = model.generate(prompts, 6, top=3)[0]
    assert tokens.shape == (3, 6) and torch.equal(tokens, again)
    assert (logprobs <= 0).all() and (entropies > 0).all()

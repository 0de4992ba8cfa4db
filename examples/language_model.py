"""A small recurrent language model from the framework's operators.

    python examples/language_model.py [--steps 30]

Trains on a synthetic language on one GPU, then generates for several requests
at once.  Per layer: input projection (``project``), gated linear recurrence
(``gated_scan``), block boundary (``block_norm``: gate, norm, residual scale,
next norm).  At the output: logits (``project`` again) and ``token_logprobs``,
whose log probabilities are the loss and whose alternatives the tokens to
choose from.  While generating, ``gated_step`` keeps every request's states in
a pool.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from nonlinear_rnn_amd import autograd as pag  # noqa: E402
from nonlinear_rnn_amd import pararnn as pr  # noqa: E402


class _Project(torch.autograd.Function):
    """u[b] = w x[b]^T on the matrix cores, channel-major; the gradients are
    plain matrix products."""

    @staticmethod
    def forward(ctx, x, w):
        ctx.save_for_backward(x, w)
        return pr.project(x, w, out_dtype=torch.bfloat16)

    @staticmethod
    def backward(ctx, du):
        x, w = ctx.saved_tensors
        B, M, T = du.shape
        rows = du.transpose(1, 2).reshape(B * T, M).contiguous()
        dx = rows @ w
        dw = rows.t().contiguous() @ x.reshape(B * T, -1)
        return dx.view(B, T, -1), dw


def project(x, w):
    return _Project.apply(x, w)


class LanguageModel(torch.nn.Module):
    """`layers` blocks of `width` channels over `vocabulary` tokens."""

    GATES = 4  # r, i, x of the recurrence, and the block's gate

    def __init__(self, vocabulary, width, layers, device="cuda", seed=0):
        super().__init__()
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, std):
            return torch.nn.Parameter((torch.randn(*shape, generator=g) * std).to(device))
        self.width, self.scale = width, 1.0 / math.sqrt(2 * layers)
        self.embedding = normal(vocabulary, width, std=1.0)
        self.head = normal(vocabulary, width, std=1.0 / math.sqrt(width))
        self.w_in = torch.nn.ParameterList(
            [normal(self.GATES * width, width, std=1.0 / math.sqrt(width)) for _ in range(layers)])
        decay = 0.9 + 0.099 * torch.rand(layers, width, generator=g)
        self.lam = torch.nn.ParameterList(
            [torch.nn.Parameter(torch.log(torch.expm1(-torch.log(a) / 8.0)).to(device)) for a in decay])
        ones = lambda: torch.nn.Parameter(torch.ones(width, device=device))  # noqa: E731
        self.w_post = torch.nn.ParameterList([ones() for _ in range(layers)])
        self.w_pre = torch.nn.ParameterList([ones() for _ in range(layers + 1)])  # one for the head

    def _planes(self, z, layer):
        """The recurrence's planes and the gate of a layer, from its normed input."""
        u = project(z, self.w_in[layer].bfloat16())
        D = self.width
        return [u[:, g * D:(g + 1) * D] for g in range(3)], u[:, 3 * D:]

    def hidden(self, tokens, resets=None, states=None):
        """The head's normed input [B][T][D] in bf16.  `states` (a list of one
        [B][D] per layer) takes the last states, for a generation to go on from."""
        x = self.embedding[tokens]
        _, z = pag.block_norm(None, x, None, self.w_pre[0])
        for layer in range(len(self.w_in)):
            u, gate = self._planes(z, layer)
            h, last = pag.gated_scan(u, self.lam[layer], resets=resets)
            if states is not None:
                states.append(last)
            x, z = pag.block_norm(h, x, self.w_post[layer], self.w_pre[layer + 1], gate=gate,
                                  scale=self.scale)
        return z

    def logits(self, z):
        """[N][V] from [N][D]: the projection with the hidden rows in the
        weights' place, so that the vocabulary is contiguous."""
        return project(self.head.bfloat16()[None], z)[0]

    def loss(self, tokens, targets, resets=None):
        """Mean negative log probability; negative targets are not scored."""
        z = self.hidden(tokens, resets)
        scores = pag.token_logprobs(self.logits(z.reshape(-1, self.width)), targets.reshape(-1))
        return -scores["logprob"].sum() / (targets >= 0).sum()

    @torch.no_grad()
    def prefill(self, pools, slot, prompt):
        """Runs a prompt [T] and leaves its states in the pools' row `slot`."""
        states = []
        z = self.hidden(prompt[None], states=states)
        for pool, state in zip(pools, states):
            pool[slot] = state[0]
        return z[0, -1]

    @torch.no_grad()
    def step(self, pools, slots, tokens):
        """One token of every request: tokens [B], slots [B] int32 (-1: idle);
        returns the head's input [B][D]."""
        x = self.embedding[tokens][:, None]
        _, z, _ = pr.block_norm(None, x, None, self.w_pre[0])
        D = self.width
        for layer in range(len(self.w_in)):
            u = pr.project(z, self.w_in[layer].bfloat16(), out_dtype=torch.bfloat16)  # [B][4 D][1]
            rows = u[:, :, 0]
            h = pr.gated_step([rows[:, g * D:(g + 1) * D] for g in range(3)], self.lam[layer],
                              pools[layer], slots=slots)
            x, z, _ = pr.block_norm(h[:, :, None], x, self.w_post[layer], self.w_pre[layer + 1],
                                    gate=u[:, 3 * D:], scale=self.scale)
        return z[:, 0]

    @torch.no_grad()
    def generate(self, prompts, new_tokens, top=5, temperature=1.0, seed=0):
        """Samples among the `top` alternatives.  prompts: 1-d token tensors of
        any lengths.  Returns (tokens [B][new_tokens], their log probabilities
        under the model, entropies)."""
        dev = self.head.device
        g = torch.Generator(dev).manual_seed(seed)
        pools = [torch.zeros((len(prompts), self.width), device=dev) for _ in self.w_in]
        slots = torch.arange(len(prompts), dtype=torch.int32, device=dev)
        z = torch.stack([self.prefill(pools, b, p) for b, p in enumerate(prompts)])
        unscored = torch.full((len(prompts),), -1, dtype=torch.int64, device=dev)
        tokens, logprobs, entropies = [], [], []
        for i in range(new_tokens):
            out = pr.token_logprobs(self.logits(z), unscored, top=top, scale=1.0 / temperature)
            pick = torch.multinomial(out["top_logprob"].exp(), 1, generator=g)
            tokens.append(out["top_index"].gather(1, pick)[:, 0])
            logprobs.append(out["top_logprob"].gather(1, pick)[:, 0])
            entropies.append(out["entropy"])
            if i + 1 < new_tokens:
                z = self.step(pools, slots, tokens[-1])
        return torch.stack(tokens, 1), torch.stack(logprobs, 1), torch.stack(entropies, 1)


def synthetic_batch(batch, length, vocabulary, seed, device="cuda"):
    """Documents that count in steps of their own: token t + 1 = token t + step.
    Returns (tokens, targets, resets); a document's last position has no target."""
    g = torch.Generator().manual_seed(seed)
    tokens = torch.empty((batch, length + 1), dtype=torch.int64)
    resets = torch.zeros((batch, length + 1), dtype=torch.bool)
    for b in range(batch):
        t = 0
        while t <= length:
            n = int(torch.randint(16, 64, (), generator=g))
            first, step = (int(torch.randint(1, vocabulary, (), generator=g)) for _ in range(2))
            n = min(n, length + 1 - t)
            tokens[b, t:t + n] = (first + (step % 7 + 1) * torch.arange(n)) % vocabulary
            resets[b, t] = True
            t += n
    targets = tokens[:, 1:].clone()
    targets[resets[:, 1:]] = -1
    return [x.contiguous().to(device) for x in (tokens[:, :-1], targets, resets[:, :-1])]


def train(model, steps, batch=8, length=256, vocabulary=256, lr=3e-3):
    opt = torch.optim.Adam(model.parameters(), lr=lr)
    losses = []
    for i in range(steps):
        loss = model.loss(*synthetic_batch(batch, length, vocabulary, seed=i))
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=30)
    a = ap.parse_args()
    model = LanguageModel(vocabulary=256, width=256, layers=2)
    losses = train(model, a.steps)
    for i in range(0, a.steps, 10):
        print(f"step {i}: loss {losses[i]:.3f}", flush=True)
    print(f"step {a.steps - 1}: loss {losses[-1]:.3f}", flush=True)
    prompts = [torch.arange(10, 10 + 3 * n, 3, device="cuda") % 256 for n in (5, 20, 33)]
    tokens, logprobs, entropies = model.generate(prompts, 8)
    for p, t, l, e in zip(prompts, tokens.tolist(), logprobs.tolist(), entropies.tolist()):
        print(f"... {p[-3:].tolist()} -> {t}  log p {sum(l):.2f}  entropy {sum(e) / len(e):.2f}")


if __name__ == "__main__":
    main()

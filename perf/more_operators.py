"""More operators of a recurrent language model, as cases that can be timed and compared.

- the gated delta rule (``step``, ``scan``, ``scan_adjoint``): a layer whose state is a matrix per head
  that stores values under keys,
    S_t = k_t a_t (S_{t-1} - b_t key_t (key_t S_{t-1})) + b_t key_t v_t,   o_t = scale query_t S_t,
  with S_t [dk][dv], a_t = exp(log_decay_t), b_t = beta_t, k_t = 0 where a new document starts;
  several value heads may share a key head;
- distillation from a teacher's most likely tokens (``distill``) and its gradient for the student's
  logits (``distill_adjoint``):
    loss = sum_e p_e (log p_e - log q_{j_e}) + r (log r - log(sum of q over the tokens not listed)),
  p the teacher's listed probabilities, r what they leave, q = softmax(scale logits);
- what a server does to logits before it samples (``adjust``): penalties for tokens that a request
  has seen, a bias for listed tokens, the mask of a grammar.

``run`` computes a case in elementary torch operations in float32, rounded once at the end; with
``own`` true it calls the package's operators.  ``exact`` computes it in float64 from the definition.
"""
import math

import torch

own = False

CHUNK = 64  # steps that the plain form takes at once
REST = 1e-6  # less than this is what rounding leaves of the teacher's listed probabilities


# ------------------------------------------------------------------- cases ---

def listed():
    return [
        # one token of a few requests of a small model: what a call costs
        dict(name="step_f32_B4_H4_64x64", op="step", B=4, Hk=4, Hv=4, dk=64, dv=64, pool=8,
             dtype="f32"),
        # one token for each of 256 requests, value heads in pairs, some of the requests idle
        dict(name="step_bf16_B256_H8_16_128x128", op="step", B=256, Hk=8, Hv=16, dk=128, dv=128,
             pool=300, dtype="bf16"),
        # a short prompt: few rows, a length that no chunk divides
        dict(name="scan_bf16_B1_T200_H8_128x128", op="scan", B=1, T=200, Hk=8, Hv=8, dk=128, dv=128,
             dtype="bf16", layout="channel", docs=0),
        # an ordinary training step on packed documents
        dict(name="scan_bf16_B8_T4096_H8_128x128", op="scan", B=8, T=4096, Hk=8, Hv=8, dk=128,
             dv=128, dtype="bf16", layout="channel", docs=512),
        # a long training sequence of a wide model, two value heads for each key head
        dict(name="scan_bf16_B4_T16384_H16_32_128x128", op="scan", B=4, T=16384, Hk=16, Hv=32,
             dk=128, dv=128, dtype="bf16", layout="channel", docs=0),
        # few heads over a very long sequence, nothing rounded
        dict(name="scan_f32_B1_T65536_H4_64x64", op="scan", B=1, T=65536, Hk=4, Hv=4, dk=64, dv=64,
             dtype="f32", layout="channel", docs=0),
        # the backward pass of the ordinary training step
        dict(name="scan_adjoint_bf16_B8_T4096_H8_128x128", op="scan_adjoint", B=8, T=4096, Hk=8,
             Hv=8, dk=128, dv=128, dtype="bf16", layout="channel", docs=512),
        # the same with nothing rounded, time-major, at sizes that no tile divides, heads shared
        dict(name="scan_adjoint_f32_B3_T1531_H2_6_80x100", op="scan_adjoint", B=3, T=1531, Hk=2, Hv=6,
             dk=80, dv=100, dtype="f32", layout="time", docs=300),
        # the loss of a student on a batch; rows of an odd vocabulary start anywhere
        dict(name="distill_bf16_N4096_V50003_k20", op="distill", N=4096, V=50003, k=20, dtype="bf16",
             tail=True, masked=False),
        # its gradient
        dict(name="distill_adjoint_bf16_N8192_V32000_k64", op="distill_adjoint", N=8192, V=32000,
             k=64, dtype="bf16", tail=True, masked=False),
        # one sampling step of 16 requests, some of them under a grammar
        dict(name="adjust_f32_N16_V65536_L2000", op="adjust", N=16, V=65536, L=2000, bias=16,
             dtype="f32", masked=True),
        # the same for many requests with long histories
        dict(name="adjust_bf16_N512_V100003_L6000", op="adjust", N=512, V=100003, L=6000, bias=0,
             dtype="bf16", masked=True),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["step", "scan", "scan", "scan_adjoint", "scan_adjoint", "distill",
                     "distill_adjoint", "adjust"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("distill", "distill_adjoint", "adjust"):
        V = _between(rng, 1000, 200000)
        N = _between(rng, 1, min(8192, 200_000_000 // V))
        masked = rng.random() < 0.5
        if op == "adjust":
            return dict(op=op, N=N, V=V, L=_between(rng, 1, max(1, min(16000, 4_000_000 // N))),
                        bias=rng.choice([0, 4, 50]), dtype=dtype, masked=masked)
        return dict(op=op, N=N, V=V, k=rng.choice([1, 5, 20, 64, 100]), dtype=dtype,
                    tail=rng.random() < 0.6, masked=masked)
    dk = rng.choice([32, 64, 128, 128, 256, rng.randint(8, 256)])
    dv = rng.choice([32, 64, 128, 128, 256, rng.randint(8, 256)])
    Hk = _between(rng, 1, 16)
    Hv = Hk * rng.choice([1, 1, 2, 3])
    if op == "step":
        B = _between(rng, 1, min(512, max(1, 80_000_000 // (Hv * dk * dv))))
        return dict(op=op, B=B, Hk=Hk, Hv=Hv, dk=dk, dv=dv, pool=B + rng.randint(0, B), dtype=dtype)
    most = (8_000_000_000 if op == "scan" else 4_000_000_000) // (Hv * dk * dv)  # steps of all rows
    T = _between(rng, 1, max(1, min(65536 if op == "scan" else 16384, most)))
    if rng.random() < 0.5:  # a multiple of 64, as training sequences are
        T = max(1, T // 64 * 64)
    B = _between(rng, 1, max(1, min(32, most // T)))
    return dict(op=op, B=B, T=T, Hk=Hk, Hv=Hv, dk=dk, dv=dv, dtype=dtype,
                layout=rng.choice(["channel", "channel", "time"]), docs=rng.choice([0, 0, 300, 2000]))


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if "V" in case:
        n = case["N"] * case["V"]
        if op == "adjust":  # logits in and out, the grammar's bits, the histories, the biases
            return dict(bytes=2 * n * e + (n // 8 if case["masked"] else 0)
                        + case["N"] * (8 * case["L"] + 12 * case["bias"] + 24), flops=4 * n)
        lists = 12 * case["N"] * case["k"]
        if op == "distill":
            return dict(bytes=n * e + lists + 12 * case["N"], flops=4 * n)
        return dict(bytes=2 * n * e + lists + 12 * case["N"], flops=5 * n)
    rows = case["B"] * case.get("T", 1)
    qk, v = rows * case["Hk"] * case["dk"], rows * case["Hv"] * case["dv"]
    gates, state = rows * case["Hv"], case["Hv"] * case["dk"] * case["dv"]
    if op == "step":  # the states in and out
        return dict(bytes=e * (2 * qk + v) + 8 * gates + 4 * v + 8 * case["B"] * state + 4 * case["B"],
                    flops=7 * rows * state)
    mask = rows if case["docs"] else 0
    if op == "scan":  # queries, keys, values and gates in, the outputs out, a state in and out
        return dict(bytes=e * (2 * qk + v) + 8 * gates + 4 * v + 8 * case["B"] * state + mask,
                    flops=7 * rows * state)
    # queries, keys, values, gates and the outputs' gradient in; gradients of each out
    return dict(bytes=2 * e * (2 * qk + v) + 16 * gates + 4 * v + 12 * case["B"] * state + mask,
                flops=21 * rows * state)


# ------------------------------------------------------------------ inputs ---

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


class _Rand:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(int(seed))

    def normal(self, *shape, std=1.0, dtype=torch.float32):
        return torch.randn(*shape, generator=self.g, device="cuda").mul_(std).to(dtype)

    def uniform(self, *shape):
        return torch.rand(*shape, generator=self.g, device="cuda")

    def whole(self, high, *shape, dtype=torch.int64, low=0):
        return torch.randint(low, high, shape, generator=self.g, device="cuda", dtype=dtype)


def _vectors(r, case, heads, size, unit):
    """[B][heads][size][T] (or without T), of unit length where they are queries or keys."""
    B, T, dtype = case["B"], case.get("T"), _DTYPES[case["dtype"]]
    x = r.normal(*((B, heads, size) if T is None else (B, T, heads, size)))
    if unit:
        x /= x.square().sum(-1, keepdim=True).sqrt()
    if T is None:
        return x.to(dtype)
    x = x.to(dtype).permute(0, 2, 3, 1)
    return x if case["layout"] == "time" else x.contiguous()


def _prepare_delta(r, case):
    B, T, Hk, Hv, dk, dv = case["B"], case.get("T"), case["Hk"], case["Hv"], case["dk"], case["dv"]
    gates = (B, Hv) if T is None else (B, Hv, T)
    rate = torch.exp(r.normal(Hv, std=1.5) - 3.5)  # a head remembers a few steps to a few thousand
    rate = rate if T is None else rate[:, None]
    s = dict(q=_vectors(r, case, Hk, dk, True), k=_vectors(r, case, Hk, dk, True),
             v=_vectors(r, case, Hv, dv, False), beta=torch.sigmoid(r.normal(*gates)),
             log_decay=-rate * torch.log1p(torch.exp(r.normal(*gates))), scale=dk ** -0.5)
    if T is None:
        slots = torch.argsort(r.uniform(case["pool"]))[:B].to(torch.int32)
        if B > 8:  # a request that has ended holds its row of the batch, but no slot
            slots[B // 2] = -1
        return s | dict(slots=slots, states=r.normal(case["pool"], Hv, dk, dv, std=0.3))
    s |= dict(h0=r.normal(B, Hv, dk, dv, std=0.1),
              resets=r.uniform(B, T) < 1.0 / case["docs"] if case["docs"] else None)
    if case["op"] == "scan_adjoint":
        go = r.normal(B, T, Hv, dv).permute(0, 2, 3, 1)
        s |= dict(go=go if case["layout"] == "time" else go.contiguous(),
                  g_last=r.normal(B, Hv, dk, dv))
    return s


def _prepare_distill(r, case):
    N, V, k = case["N"], case["V"], case["k"]
    dtype = _DTYPES[case["dtype"]]
    x = r.normal(N, V, std=2.5)
    if case["masked"]:  # a grammar allows a part of the vocabulary, and in one row very few tokens
        x.masked_fill_(r.uniform(N, V) < 0.6, -math.inf)
        if N > 4:
            x[N // 2, 3:] = -math.inf
            x[N // 2, :3] = 0.5
    index, logprob = [], []
    for rows in x.split(max(1, 50_000_000 // V)):  # the teacher agrees with the student in part
        t = torch.log_softmax(0.8 * rows + r.normal(*rows.shape, std=1.5), -1)
        value, at = t.topk(min(k, V), -1)
        index.append(torch.where(torch.isneginf(value), -1, at))
        logprob.append(value)
    index, logprob = torch.cat(index).contiguous(), torch.cat(logprob).contiguous()
    index[N // 3::7] = -1  # positions that the teacher has not scored
    s = dict(logits=x.to(dtype), index=index, logprob=logprob)
    if case["op"] == "distill_adjoint":
        out = _plain_distill(s | dict(case=case))
        s |= dict(lse=out["lse"], log_rest=out["log_rest"], g_loss=r.uniform(N) / N * 100)
    return s


def _prepare_adjust(r, case):
    N, V, L, M = case["N"], case["V"], case["L"], case["bias"]
    # texts repeat themselves: few tokens often, most never
    tokens = (V * r.uniform(N, L) ** 4).long().clamp(max=V - 1)
    lengths = (L * r.uniform(N)).to(torch.int32) + 1
    s = dict(logits=r.normal(N, V, std=2.5).to(_DTYPES[case["dtype"]]), tokens=tokens, lengths=lengths,
             prompt=(lengths * r.uniform(N)).to(torch.int32), repetition=1.0 + 0.3 * r.uniform(N),
             presence=r.uniform(N), frequency=0.2 * r.uniform(N), bias=None, allowed=None, rows=None)
    if M:
        index = r.whole(V, N, M)
        index[:, M // 2] = -1
        s["bias"] = (index, r.normal(N, M, std=3.0))
    if case["masked"]:  # a few grammars, each for many requests; some requests have none
        R = min(N, 40)
        words = r.whole(2 ** 31, R, (V + 31) // 32, dtype=torch.int64, low=-2 ** 31)
        s |= dict(allowed=words.to(torch.int32), rows=r.whole(R, N, dtype=torch.int32, low=-1))
    return s


def prepare(case, seed):
    r = _Rand(seed)
    if case["op"] == "adjust":
        s = _prepare_adjust(r, case)
    elif "V" in case:
        s = _prepare_distill(r, case)
    else:
        s = _prepare_delta(r, case)
    return s | dict(case=case)


# ------------------------------------------------------------- plain forms ---

def _plain_step(s):
    group = s["v"].shape[1] // s["q"].shape[1]
    q, k = (x.float().repeat_interleave(group, 1) for x in (s["q"], s["k"]))
    slots, old = s["slots"].long(), s["states"]
    live = (slots >= 0)[:, None, None, None]
    S = torch.exp(s["log_decay"])[..., None, None] * old[slots.clamp(min=0)]
    write = s["beta"][..., None] * (s["v"].float() - (k[..., None] * S).sum(2))
    S = S + k[..., None] * write[:, :, None]
    o = s["scale"] * (q[..., None] * S).sum(2)
    keep = torch.cat([old, old[:1]])  # idle rows write to a row past the pool
    states = keep.index_copy(0, torch.where(slots >= 0, slots, old.shape[0]), S)[:-1]
    return torch.where(live[..., 0], o, torch.zeros(()).to(o)), states


def _inverse(A):
    """(I + A)^-1 of strictly lower triangular A: blocks of the diagonal joined two by two."""
    n = A.shape[-1]
    at = torch.arange(n, device=A.device)
    X = torch.eye(n, device=A.device).expand_as(A)
    size = 1
    while size < n:
        block = at // size
        pair = (block[:, None] == block[None, :] + 1) & (block[:, None] % 2 == 1)
        X = X - X @ (A * pair) @ X
        size *= 2
    return X


def _plain_scan(q, k, v, beta, log_decay, h0, resets, scale):
    """A chunk of steps at once: within it, what the steps write solves a triangular system."""
    B, Hv, dv, T = v.shape
    N = -(-T // CHUNK)
    pad = N * CHUNK - T

    def chunks(x):  # [B][H][d][T] to [B][Hv][N][CHUNK][d]
        x = torch.nn.functional.pad(x, (0, pad)).unflatten(-1, (N, CHUNK)).permute(0, 1, 3, 4, 2)
        return x.repeat_interleave(Hv // x.shape[1], 1)
    q, k, v, beta, g = chunks(q), chunks(k), chunks(v), chunks(beta[:, :, None]), chunks(log_decay[:, :, None])
    G = torch.cumsum(g.double(), -2)  # differences of far sums
    at = torch.arange(CHUNK, device=v.device)
    if resets is None:
        same = torch.ones((), dtype=torch.bool, device=v.device)
        from_start, to_end = same, same
    else:  # the document of each step, counted from the chunk's start
        doc = torch.cumsum(torch.nn.functional.pad(resets, (0, pad)).long().unflatten(-1, (N, CHUNK)), -1)
        doc = doc[:, None, ..., None]
        same, from_start, to_end = doc == doc.transpose(-1, -2), doc == 0, doc == doc[..., -1:, :]

    def factor(keep, x):
        return torch.where(keep, torch.exp(torch.where(keep, x, 0.0)), 0.0).float()
    D = factor(same & (at[:, None] >= at[None, :]), G - G.transpose(-1, -2))
    first, last = factor(from_start, G), factor(to_end, G[..., -1:, :] - G)
    across = (first[..., -1:, :] if resets is not None else torch.exp(G[..., -1:, :]).float())
    X = _inverse(beta * (k @ k.transpose(-1, -2)) * D * (at[:, None] > at[None, :]))
    U, W = X @ (beta * v), X @ (beta * first * k)
    P = scale * (q @ k.transpose(-1, -2)) * D
    Q, K = scale * first * q, (last * k).transpose(-1, -2)
    S, out = h0, []
    for n in range(N):
        new = U[:, :, n] - W[:, :, n] @ S
        out.append(Q[:, :, n] @ S + P[:, :, n] @ new)
        S = across[:, :, n] * S + K[:, :, n] @ new
    o = torch.stack(out, 2).permute(0, 1, 4, 2, 3).flatten(-2)[..., :T]
    return o, S


def _plain_scan_case(s):
    o, S = _plain_scan(s["q"].float(), s["k"].float(), s["v"].float(), s["beta"], s["log_decay"], s["h0"],
                       s["resets"], s["scale"])
    return o.contiguous(), S


def _plain_scan_adjoint(s):
    names = ("q", "k", "v", "beta", "log_decay", "h0")
    leaves = [s[n].float().detach().requires_grad_(True) for n in names]
    o, S = _plain_scan(*leaves, s["resets"], s["scale"])
    grads = torch.autograd.grad([o, S], leaves, [s["go"], s["g_last"]])
    return {"d" + n: g.to(s[n].dtype).contiguous() for n, g in zip(names, grads)}


def _plain_distill(s):
    x = s["case"].get("scale", 1.0) * s["logits"].float()
    index, used = s["index"].clamp(min=0), s["index"] >= 0
    m = x.max(-1, keepdim=True).values
    m = torch.where(torch.isneginf(m), 0.0, m)
    e = torch.exp(x - m)
    lse = (m + torch.log(e.sum(-1, keepdim=True)))
    hit = torch.zeros(x.shape[0], x.shape[1] + 1, dtype=torch.bool, device=x.device)
    hit.scatter_(1, torch.where(used, s["index"], x.shape[1]), True)
    rest = torch.where(hit[:, :-1], 0.0, e).sum(-1, keepdim=True)
    log_rest = torch.log(rest) + m - lse
    lp = torch.where(used, s["logprob"], -math.inf)
    p = torch.exp(lp)
    term = p * (lp - (x.gather(1, index) - lse))
    loss = torch.where(p > 0, term, 0.0).sum(-1)
    if s["case"]["tail"]:
        r = 1.0 - p.sum(-1)
        term = r * (torch.log(r) - log_rest[:, 0])
        loss = loss + torch.where(r >= REST, term, 0.0)
    return dict(loss=loss, lse=lse[:, 0], log_rest=log_rest[:, 0])


def _plain_distill_adjoint(s):
    x, scale = s["logits"].float(), s["case"].get("scale", 1.0)
    V = x.shape[1]
    used = s["index"] >= 0
    q = torch.exp(scale * x - s["lse"][:, None])
    p = torch.where(used, torch.exp(s["logprob"]), 0.0)
    total = p.sum(-1, keepdim=True)
    if s["case"]["tail"]:
        r = 1.0 - total
        r = torch.where(r >= REST, r, 0.0)
        hit = torch.zeros(x.shape[0], V + 1, dtype=torch.bool, device=x.device)
        hit.scatter_(1, torch.where(used, s["index"], V), True)
        share = torch.where(r > 0, r * torch.exp(-s["log_rest"][:, None]), 0.0)
        outside = torch.where(q > 0, q * (total + r - share), 0.0)
        grad = torch.where(hit[:, :-1], q * (total + r), outside)
    else:
        grad = q * total
    grad.scatter_add_(1, s["index"].clamp(min=0), -p)
    return (scale * s["g_loss"][:, None] * grad).to(s["logits"].dtype)


def _plain_adjust(s):
    x = s["logits"].float()
    N, V = x.shape
    tokens = s["tokens"]
    at = torch.arange(tokens.shape[1], device=x.device)
    real = at < s["lengths"][:, None]
    new = real & (at >= s["prompt"][:, None])
    count, seen = torch.zeros(N, V, device=x.device), torch.zeros(N, V, device=x.device)
    count.scatter_add_(1, tokens, new.float())
    seen.scatter_add_(1, tokens, real.float())
    rep = s["repetition"][:, None]
    x = torch.where(seen > 0, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0).float()
    if s["bias"] is not None:
        index, value = s["bias"]
        used = index >= 0
        # the last of a token's entries counts
        order = torch.arange(1, index.shape[1] + 1, device=x.device).expand_as(index)
        entry = torch.zeros(N, V + 1, dtype=torch.int64, device=x.device)
        entry.scatter_reduce_(1, torch.where(used, index, V), order, "amax")
        entry = entry[:, :V]
        x = x + torch.where(entry > 0, value.gather(1, (entry - 1).clamp(min=0)), 0.0)
    if s["allowed"] is not None:
        j = torch.arange(V, device=x.device)
        rows = s["rows"].long()
        word = s["allowed"][rows.clamp(min=0)][:, j // 32]
        allowed = ((word >> (j % 32).int()) & 1) != 0
        x = torch.where(allowed | (rows < 0)[:, None], x, -math.inf)
    return x.to(s["logits"].dtype)


# --------------------------------------------------------------------- run ---

def _own_run(s):
    from nonlinear_rnn_amd import pararnn as pr

    op = s["case"]["op"]
    if op == "step":
        o = pr.delta_step(s["q"], s["k"], s["v"], s["beta"], s["log_decay"], s["states"],
                          slots=s["slots"], scale=s["scale"])
        return o, s["states"]
    if op == "scan":
        return pr.delta_scan(s["q"], s["k"], s["v"], s["beta"], s["log_decay"], s["h0"],
                             scale=s["scale"], resets=s["resets"])
    if op == "scan_adjoint":
        return pr.delta_scan_adjoint(s["q"], s["k"], s["v"], s["beta"], s["log_decay"], s["h0"], s["go"],
                                     g_last=s["g_last"], scale=s["scale"], resets=s["resets"])
    if op == "distill":
        return pr.distill_top(s["logits"], s["index"], s["logprob"], tail=s["case"]["tail"])
    if op == "distill_adjoint":
        return pr.distill_top_adjoint(s["logits"], s["index"], s["logprob"], s["lse"], s["log_rest"],
                                      s["g_loss"], tail=s["case"]["tail"])
    return pr.adjust_logits(s["logits"], tokens=s["tokens"], lengths=s["lengths"], prompt=s["prompt"],
                            repetition=s["repetition"], presence=s["presence"],
                            frequency=s["frequency"], bias=s["bias"], allowed=s["allowed"],
                            allowed_rows=s["rows"])


def run(s):
    if own:
        return _own_run(s)
    op = s["case"]["op"]
    if op == "step":  # the states are updated in place, as a server keeps them
        o, states = _plain_step(s)
        s["states"].copy_(states)
        return o, s["states"]
    if op == "scan":
        return _plain_scan_case(s)
    if op == "scan_adjoint":
        return _plain_scan_adjoint(s)
    if op == "distill":
        return _plain_distill(s)
    if op == "distill_adjoint":
        return _plain_distill_adjoint(s)
    return _plain_adjust(s)


# ------------------------------------------------------------------- exact ---

def _advance(S, a, k, v, b):
    """One step of states [rows][dk][dv]; a, b [rows]: (decayed state, what is written, new state)."""
    S = a[:, None, None] * S
    w = b[:, None] * (v - torch.bmm(k[:, None], S)[:, 0])
    return S, w, torch.baddbmm(S, k[:, :, None], w[:, None])


def _exact_delta(s, adjoint):
    B, Hv, dv, T = s["v"].shape
    Hk, dk = s["q"].shape[1:3]

    def by_step(x, heads):  # [T][B Hv][d]
        x = x.double().unsqueeze(2) if x.dim() == 3 else x.double()
        return x.repeat_interleave(Hv // heads, 1).permute(3, 0, 1, 2).reshape(T, B * Hv, -1).contiguous()
    q, k, v = by_step(s["q"], Hk), by_step(s["k"], Hk), by_step(s["v"], Hv)
    b, a = by_step(s["beta"], Hv)[..., 0], torch.exp(by_step(s["log_decay"], Hv))[..., 0]
    if s["resets"] is not None:
        a = a * (~s["resets"]).double().t().repeat_interleave(Hv, 1)
    S = s["h0"].double().reshape(B * Hv, dk, dv)
    span = max(1, int(math.sqrt(T)))
    kept, o = [], torch.empty(T, B * Hv, dv, dtype=torch.float64, device=S.device) if not adjoint else None
    for t in range(T):
        if adjoint and t % span == 0:
            kept.append(S)
        S = _advance(S, a[t], k[t], v[t], b[t])[2]
        if not adjoint:
            o[t] = s["scale"] * torch.bmm(q[t][:, None], S)[:, 0]
    if not adjoint:
        return o.view(T, B, Hv, dv).permute(1, 2, 3, 0), S.view(B, Hv, dk, dv)
    go = by_step(s["go"], Hv) * s["scale"]
    gS = s["g_last"].double().reshape(B * Hv, dk, dv)
    gq, gk, gv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    gb, gl = torch.empty_like(b), torch.empty_like(a)
    for first in range((T - 1) // span * span, -1, -span):
        states = [kept[first // span]]
        for t in range(first, min(T, first + span) - 1):
            states.append(_advance(states[-1], a[t], k[t], v[t], b[t])[2])
        for t in range(min(T, first + span) - 1, first - 1, -1):
            decayed, w, after = _advance(states[t - first], a[t], k[t], v[t], b[t])
            gq[t] = torch.bmm(after, go[t][:, :, None])[:, :, 0]
            gS = torch.baddbmm(gS, q[t][:, :, None], go[t][:, None])
            gw = torch.bmm(k[t][:, None], gS)[:, 0]  # of what the step writes
            miss = v[t] - torch.bmm(k[t][:, None], decayed)[:, 0]
            gb[t] = (gw * miss).sum(-1)
            gv[t] = b[t][:, None] * gw
            gk[t] = torch.bmm(gS, w[:, :, None])[:, :, 0] - torch.bmm(decayed, gv[t][:, :, None])[:, :, 0]
            gS = torch.baddbmm(gS, k[t][:, :, None], gv[t][:, None], alpha=-1)
            gl[t] = (gS * decayed).sum((1, 2))
            gS = a[t][:, None, None] * gS

    def back(x, heads):
        x = x.view(T, B, heads, Hv // heads, -1).sum(3)
        return x.permute(1, 2, 3, 0)
    return dict(dq=back(gq, Hk), dk=back(gk, Hk), dv=back(gv, Hv), dbeta=back(gb, Hv)[:, :, 0],
                dlog_decay=back(gl, Hv)[:, :, 0], dh0=gS.view(B, Hv, dk, dv))


def _exact_step(s):
    B, Hv, dv = s["v"].shape
    group = Hv // s["q"].shape[1]
    states = s["states"].double()
    o = torch.zeros(B, Hv, dv, dtype=torch.float64, device=states.device)
    for row, slot in enumerate(s["slots"].tolist()):
        if slot < 0:
            continue
        q, k = (x[row].double().repeat_interleave(group, 0) for x in (s["q"], s["k"]))
        S = _advance(states[slot], torch.exp(s["log_decay"][row].double()), k, s["v"][row].double(),
                     s["beta"][row].double())[2]
        states[slot] = S
        o[row] = s["scale"] * torch.bmm(q[:, None], S)[:, 0]
    return o, states


def _exact_distill(s, adjoint):
    out = dict(loss=[], lse=[], log_rest=[], grad=[])
    V = s["logits"].shape[1]
    for n in range(0, len(s["logits"]), 256):
        x, index, lp = (s[name][n:n + 256] for name in ("logits", "index", "logprob"))
        x, p = x.double(), torch.where(index >= 0, torch.exp(lp.double()), 0.0)
        logq = torch.log_softmax(x, -1)
        outside = torch.ones_like(x)
        rows = torch.arange(len(x), device=x.device)[:, None].expand_as(index)
        outside[rows[index >= 0], index[index >= 0]] = 0.0
        rest = (outside * torch.exp(logq)).sum(-1)
        r = 1.0 - p.sum(-1)
        r = torch.where(r < REST, 0.0, r) if s["case"]["tail"] else torch.zeros_like(r)
        if adjoint:  # from the log probabilities' gradients, through the softmax
            g = torch.zeros_like(x)
            g.index_put_((rows.reshape(-1), index.clamp(min=0).reshape(-1)), -p.reshape(-1), accumulate=True)
            g -= torch.where(r > 0, r / rest, 0.0)[:, None] * outside * torch.exp(logq)
            grad = g - torch.exp(logq) * g.sum(-1, keepdim=True)
            out["grad"].append(s["g_loss"][n:n + 256].double()[:, None] * grad)
            continue
        out["lse"].append(torch.logsumexp(x, -1))
        out["log_rest"].append(torch.log(rest))
        at = logq.gather(1, index.clamp(min=0))
        loss = torch.where(p > 0, p * (lp.double() - at), 0.0).sum(-1)
        out["loss"].append(loss + torch.where(r > 0, r * (torch.log(r) - torch.log(rest)), 0.0))
    return torch.cat(out["grad"]) if adjoint else {n: torch.cat(out[n]) for n in ("loss", "lse", "log_rest")}


def _exact_adjust(s):
    x = s["logits"].double()
    N, V = x.shape
    lengths, prompts = s["lengths"].tolist(), s["prompt"].tolist()
    rows = None if s["rows"] is None else s["rows"].tolist()
    rep, presence, frequency = (s[n].double().tolist() for n in ("repetition", "presence", "frequency"))
    place = torch.arange(32, device=x.device)
    for n in range(N):
        seen = torch.unique(s["tokens"][n, :lengths[n]])
        x[n, seen] = torch.where(x[n, seen] < 0, x[n, seen] * rep[n], x[n, seen] / rep[n])
        new, times = torch.unique(s["tokens"][n, prompts[n]:lengths[n]], return_counts=True)
        x[n, new] -= presence[n] + frequency[n] * times.double()
        if s["bias"] is not None:
            last = {j: v for j, v in zip(s["bias"][0][n].tolist(), s["bias"][1][n].tolist()) if j >= 0}
            x[n, list(last)] += torch.tensor(list(last.values()), dtype=torch.float64, device=x.device)
        if rows is not None and rows[n] >= 0:
            bits = (s["allowed"][rows[n]].long()[:, None] >> place & 1).reshape(-1)[:V]
            x[n].masked_fill_(bits == 0, -math.inf)
    return x


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("scan", "scan_adjoint"):
        return _exact_delta(s, op == "scan_adjoint")
    if op == "step":
        return _exact_step(s)
    if op in ("distill", "distill_adjoint"):
        return _exact_distill(s, op == "distill_adjoint")
    return _exact_adjust(s)

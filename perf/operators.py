"""The operators of a recurrent language model, as cases that can be timed and compared.

Three operators that meet in every layer and at the output of such a model:

- the gated linear recurrence (``step``, ``scan``, ``scan_adjoint``):
    l = -power softplus(lam) sigmoid(u_r),  a = exp(l),
    h_t = k_t a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(u_i) u_x,
  k_t = 0 where a new document starts, 1 elsewhere;
- the block boundary (``block``, ``block_adjoint``): the gated states, normed, scaled and added to
  the residual stream, and the norm in front of the next block:
    v = h silu(g),  y = x + scale v rstd(v) w_post,  z = y rstd(y) w_pre;
- log probabilities of given tokens with entropy and top alternatives (``score``), and their
  gradient (``score_adjoint``).

``run`` computes a case in elementary torch operations in float32, rounded once at the end; with
``own`` true it calls the package's operators.  ``exact`` computes it in float64 from the definition.
"""
import math

import torch

own = False

POWER = 8.0
SCALE = 0.25
EPS = 1e-6


# ------------------------------------------------------------------- cases ---

def listed():
    return [
        # one generated token for each of 64 requests, their states in a pool with idle slots
        dict(name="step_f32_B64_D1024", op="step", B=64, D=1024, pool=96, dtype="f32"),
        # few channels over a very long sequence: the work has to be split along time
        dict(name="scan_f32_B1_T262144_D64", op="scan", B=1, T=262144, D=64, dtype="f32",
             layout="channel", docs=0),
        # a long training sequence with every channel of a wide model
        dict(name="scan_bf16_B4_T16384_D4096", op="scan", B=4, T=16384, D=4096, dtype="bf16",
             layout="channel", docs=0),
        # the backward pass of an ordinary training step on packed documents
        dict(name="scan_adjoint_bf16_B8_T4096_D1024", op="scan_adjoint", B=8, T=4096, D=1024,
             dtype="bf16", layout="channel", docs=512),
        # the block boundary while generating: one token for each of 64 requests
        dict(name="block_bf16_B64_T1_D1024", op="block", B=64, T=1, D=1024, dtype="bf16",
             stream="bf16"),
        # the block boundary of an ordinary training step
        dict(name="block_bf16_B8_T4096_D1024", op="block", B=8, T=4096, D=1024, dtype="bf16",
             stream="f32"),
        # its backward pass at the widest configuration
        dict(name="block_adjoint_bf16_B16_T2048_D4096", op="block_adjoint", B=16, T=2048, D=4096,
             dtype="bf16", stream="f32"),
        # the same with nothing rounded, at sizes that no tile divides
        dict(name="block_adjoint_f32_B3_T1531_D2000", op="block_adjoint", B=3, T=1531, D=2000,
             dtype="f32", stream="f32"),
        # scores of one sampled token for each of 16 requests, some tokens masked by a grammar
        dict(name="score_f32_N16_V65536_k20", op="score", N=16, V=65536, k=20, dtype="f32",
             masked=True),
        # scores of a batch of prompts; rows of an odd vocabulary start anywhere
        dict(name="score_bf16_N4096_V50003_k8", op="score", N=4096, V=50003, k=8, dtype="bf16",
             masked=False),
        # the loss gradient of a training step
        dict(name="score_adjoint_bf16_N8192_V32000", op="score_adjoint", N=8192, V=32000,
             dtype="bf16", masked=False),
        # a policy gradient: log probabilities and entropy of masked samples, nothing rounded
        dict(name="score_adjoint_f32_N1000_V100003", op="score_adjoint", N=1000, V=100003,
             dtype="f32", masked=True),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["step", "scan", "scan", "scan_adjoint", "block", "block_adjoint", "score",
                     "score_adjoint"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "step":
        B = _between(rng, 1, 512)
        return dict(op=op, B=B, D=_between(rng, 64, 8192), pool=B + rng.randint(0, B), dtype=dtype)
    if op in ("score", "score_adjoint"):
        V = _between(rng, 1000, 200000)
        N = _between(rng, 1, min(8192, 200_000_000 // V))
        case = dict(op=op, N=N, V=V, dtype=dtype, masked=rng.random() < 0.5)
        return {**case, "k": rng.choice([0, 1, 5, 8, 20, 50])} if op == "score" else case
    D = _between(rng, 64, 4096) if rng.random() < 0.5 else 64 * _between(rng, 1, 64)
    most = 100_000_000 if op != "scan" else 200_000_000  # values of one plane
    T = _between(rng, 1, min(8192 if op.startswith("block") else 262144, most // D))
    if rng.random() < 0.5:  # a multiple of 64, as training sequences are
        T = max(1, T // 64 * 64)
    B = _between(rng, 1, max(1, min(64, most // (D * T))))
    case = dict(op=op, B=B, T=T, D=D, dtype=dtype)
    if op in ("block", "block_adjoint"):
        return {**case, "stream": rng.choice(["f32", "bf16"])}
    return {**case, "layout": rng.choice(["channel", "channel", "time"]),
            "docs": rng.choice([0, 0, 300, 2000])}


def _elements(case):
    if "V" in case:
        return case["N"] * case["V"]
    return case["B"] * case["D"] * case.get("T", 1)


def work(case):
    n, e = _elements(case), 2 if case["dtype"] == "bf16" else 4
    s = 2 if case.get("stream") == "bf16" else 4
    op = case["op"]
    if op == "step":  # three projections and the state in; the state and the output out
        return dict(bytes=n * (3 * e + 12) + 4 * case["D"] + 4 * case["B"], flops=25 * n)
    if op in ("scan", "scan_adjoint"):
        rows = case["B"] * case["D"]
        mask = case["B"] * case["T"] if case["docs"] else 0
        if op == "scan":  # three projections in, the states out
            return dict(bytes=n * (3 * e + 4) + 8 * rows + 4 * case["D"] + mask, flops=25 * n)
        # three projections, the states and their gradient in; three gradients out
        return dict(bytes=n * (6 * e + 8) + 8 * rows + 8 * case["D"] + mask, flops=45 * n)
    if op == "block":  # states, gate and stream in; stream and normed stream out
        return dict(bytes=n * (4 + e + 2 * s + 2) + 8 * case["D"] + 8 * case["B"] * case["T"],
                    flops=18 * n)
    if op == "block_adjoint":  # states, gate, stream and two gradients in; three gradients out
        return dict(bytes=n * (8 + 2 * e + 3 * s + 2) + 16 * case["D"] + 8 * case["B"] * case["T"],
                    flops=45 * n)
    if op == "score":
        return dict(bytes=n * e + case["N"] * (8 + 12 + 12 * case["k"]), flops=6 * n)
    return dict(bytes=2 * n * e + case["N"] * (8 + 20), flops=8 * n)


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

    def whole(self, high, *shape, dtype=torch.int64):
        return torch.randint(0, high, shape, generator=self.g, device="cuda", dtype=dtype)


def _lam(r, D):
    """Decays as such models start with: exp(-power softplus(lam)) over (0.9, 0.999)."""
    a = 0.9 + 0.099 * r.uniform(D)
    return torch.log(torch.expm1(-torch.log(a) / POWER))


def _planes(r, n, case, dtype, std=1.0):
    B, T, D = case["B"], case["T"], case["D"]
    if case.get("layout") == "time":
        return [r.normal(B, T, D, std=std, dtype=dtype).transpose(1, 2) for _ in range(n)]
    return [r.normal(B, D, T, std=std, dtype=dtype) for _ in range(n)]


def prepare(case, seed):
    r = _Rand(seed)
    op, dtype = case["op"], _DTYPES[case["dtype"]]
    s = dict(case=case)
    if op == "step":
        B, D, pool = case["B"], case["D"], case["pool"]
        slots = torch.argsort(r.uniform(pool))[:B].to(torch.int32)
        if B > 8:  # a request that has ended holds its row of the batch, but no slot
            slots[B // 2] = -1
        u = r.normal(B, 3 * D, dtype=dtype)
        s |= dict(u=[u[:, g * D:(g + 1) * D] for g in range(3)], lam=_lam(r, D), slots=slots,
                  states=r.normal(pool, D, std=0.5))
    elif op in ("scan", "scan_adjoint"):
        B, T, D = case["B"], case["T"], case["D"]
        s |= dict(u=_planes(r, 3, case, dtype), lam=_lam(r, D), h0=r.normal(B, D, std=0.1),
                  resets=r.uniform(B, T) < 1.0 / case["docs"] if case["docs"] else None)
        if op == "scan_adjoint":
            h = _plain_scan(s)[0]
            s["h"] = h.transpose(1, 2).contiguous().transpose(1, 2) if case["layout"] == "time" else h
            s["gh"] = _planes(r, 1, case, torch.float32)[0]
    elif op in ("block", "block_adjoint"):
        B, T, D = case["B"], case["T"], case["D"]
        stream = _DTYPES[case["stream"]]
        s |= dict(h=r.normal(B, D, T, std=0.5), gate=r.normal(B, D, T, dtype=dtype),
                  x=r.normal(B, T, D, std=2.0, dtype=stream),
                  w_post=1.0 + r.normal(D, std=0.1), w_pre=1.0 + r.normal(D, std=0.1))
        if op == "block_adjoint":
            s["rstd"] = _plain_block(s)[2]
            s["gy"] = r.normal(B, T, D, dtype=stream)
            s["gz"] = r.normal(B, T, D, dtype=torch.bfloat16)
    else:
        N, V = case["N"], case["V"]
        x = r.normal(N, V, std=2.5)
        x += r.normal(N, 1, std=3.0)
        tokens = r.whole(V, N)
        if case["masked"]:  # a grammar allows a part of the vocabulary, and in one row nothing
            x.masked_fill_(r.uniform(N, V) < 0.6, -math.inf)
            if N > 4:
                x[N // 2] = -math.inf
        tokens[N // 3::7] = -1  # positions of the prompt that nothing scores
        s |= dict(logits=x.to(dtype), tokens=tokens)
        if op == "score_adjoint":
            out = _plain_score(s, 0)
            s |= dict(lse=out["lse"], entropy=out["entropy"])
            s |= dict(g_logprob=r.normal(N), g_entropy=r.normal(N, std=0.1), g_lse=r.normal(N, std=0.1))
    return s


# ------------------------------------------------------------- plain forms ---

def _gates(s):
    """log decay, decay, input gain, input gate and value, in float32."""
    ur, ui, ux = (p.float() for p in s["u"])
    lam = torch.log1p(torch.exp(s["lam"]))  # softplus; lam is below zero here
    lam = lam if ur.dim() == 2 else lam[:, None]
    l = -POWER * lam * torch.sigmoid(ur)
    return l, torch.exp(l), torch.sqrt(-torch.expm1(2 * l)), torch.sigmoid(ui), ux


def _doubling(a, b):
    """x_t = a_t x_{t-1} + b_t from x_0 = 0: pairs of spans joined, log2(T) times over the planes."""
    T, span = a.shape[-1], 1
    while span < T:
        b = torch.cat([b[..., :span], b[..., span:] + a[..., span:] * b[..., :-span]], -1)
        a = torch.cat([a[..., :span], a[..., span:] * a[..., :-span]], -1)
        span *= 2
    return b


def _keep(s, a):
    return a if s["resets"] is None else a * (~s["resets"][:, None, :]).float()


def _plain_step(s):
    _, a, gain, i, x = _gates(s)
    old, slots = s["states"], s["slots"].long()
    live = (slots >= 0)[:, None]
    at = slots.clamp(min=0)
    new = torch.where(live, a * old[at] + gain * i * x, torch.zeros(()).to(a))
    keep = torch.cat([old, old[:1]])  # idle rows write to a row past the pool
    states = keep.index_copy(0, torch.where(slots >= 0, slots, old.shape[0]), new)[:-1]
    return new, states


def _plain_scan(s):
    _, a, gain, i, x = _gates(s)
    a, b = _keep(s, a).contiguous(), (gain * i * x).contiguous()
    b[..., 0] += a[..., 0] * s["h0"]
    h = _doubling(a, b)
    return h, h[..., -1].contiguous()


def _plain_scan_adjoint(s):
    dtype = s["u"][0].dtype
    l, a, gain, i, x = _gates(s)
    kept = _keep(s, a)
    # lambda_t = gh_t + kept_{t+1} lambda_{t+1}, backwards in time
    after = torch.cat([kept[..., 1:], torch.zeros_like(kept[..., :1])], -1)
    g = _doubling(after.flip(-1), s["gh"].flip(-1)).flip(-1)
    before = torch.cat([s["h0"][..., None], s["h"][..., :-1]], -1)
    gx = g * gain * i
    gi = g * gain * x * i * (1 - i)
    gl = g * (kept * before - a * a / gain * i * x)
    sig = torch.sigmoid(s["u"][0].float())
    lam = s["lam"]
    glam = (gl * sig).sum((0, 2)) * -POWER * torch.sigmoid(lam)
    return dict(du=[(gl * l * (1 - sig)).to(dtype), gi.to(dtype), gx.to(dtype)], dlam=glam,
                dh0=(kept * g)[..., 0].contiguous())


def _plain_block(s):
    h, g = s["h"].transpose(1, 2), s["gate"].float().transpose(1, 2)
    v = h * g * torch.sigmoid(g)
    r1 = torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    y = s["x"].float() + SCALE * v * r1 * s["w_post"]
    r2 = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS)
    z = y * r2 * s["w_pre"]
    return y.to(s["x"].dtype), z.bfloat16(), torch.stack([r1[..., 0], r2[..., 0]])


def _plain_block_adjoint(s):
    h, g = s["h"].transpose(1, 2), s["gate"].float().transpose(1, 2)
    r1, r2 = s["rstd"][0][..., None], s["rstd"][1][..., None]
    sig = torch.sigmoid(g)
    v = h * g * sig
    n1 = v * r1
    n2 = (s["x"].float() + SCALE * n1 * s["w_post"]) * r2
    gz = s["gz"].float()
    q = gz * s["w_pre"]
    gy = s["gy"].float() + r2 * (q - n2 * (q * n2).mean(-1, keepdim=True))
    p = SCALE * gy * s["w_post"]
    gv = r1 * (p - n1 * (p * n1).mean(-1, keepdim=True))
    return dict(dx=gy.to(s["x"].dtype), dh=(gv * g * sig).transpose(1, 2).contiguous(),
                dgate=(gv * h * sig * (1 + g * (1 - sig))).transpose(1, 2).contiguous().to(s["gate"].dtype),
                dw_post=(SCALE * gy * n1).sum((0, 1)), dw_pre=(gz * n2).sum((0, 1)))


def _plain_score(s, k):
    x, tokens = s["logits"].float(), s["tokens"]
    N, V = x.shape
    m = x.max(-1, keepdim=True).values
    none = torch.isneginf(m)
    d = x - torch.where(none, torch.zeros_like(m), m)
    e = torch.exp(d)
    total = e.sum(-1, keepdim=True)
    log_total = torch.where(none, -math.inf, torch.log(total))
    lse = log_total + torch.where(none, torch.zeros_like(m), m)
    # entropy = log(sum e) - sum(e d) / sum(e); a masked token adds nothing
    mean = torch.where(e > 0, e * d, torch.zeros_like(e)).sum(-1, keepdim=True) / total
    entropy = torch.where(none, torch.zeros_like(m), log_total - mean)[:, 0]
    logprob = (d.gather(1, tokens.clamp(min=0)[:, None]) - torch.where(none, torch.zeros_like(m), log_total))[:, 0]
    out = dict(logprob=torch.where(tokens >= 0, logprob, torch.zeros_like(logprob)), entropy=entropy,
               lse=lse[:, 0])
    if k:  # the largest k; of equal ones the lowest index first: one order of whole numbers
        bits = x.view(torch.int32).long()
        bits = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
        key = bits * 2 ** 32 + (V - 1 - torch.arange(V, device=x.device))
        top = V - 1 - (key.topk(k, -1).values & (2 ** 32 - 1))
        value = d.gather(1, top) - log_total
        out["top_index"] = torch.where(torch.isneginf(x.gather(1, top)), -1, top)
        out["top_logprob"] = torch.where(out["top_index"] < 0, -math.inf, value)
    return out


def _plain_score_adjoint(s):
    x, tokens = s["logits"].float(), s["tokens"]
    lse, entropy = s["lse"][:, None], s["entropy"][:, None]
    none = torch.isneginf(lse)
    logp = x - torch.where(none, torch.zeros_like(lse), lse)
    p = torch.where(none, torch.zeros_like(x), torch.exp(logp))
    glp = torch.where(tokens >= 0, s["g_logprob"], torch.zeros_like(s["g_logprob"]))[:, None]
    coefficient = s["g_lse"][:, None] - glp - s["g_entropy"][:, None] * (logp + entropy)
    grad = torch.where(p > 0, p * coefficient, torch.zeros_like(p))
    hit = torch.where(none, torch.zeros_like(glp), glp)
    grad.scatter_add_(1, tokens.clamp(min=0)[:, None], hit)
    return grad.to(s["logits"].dtype)


# --------------------------------------------------------------------- run ---

def _own_run(s):
    from nonlinear_rnn_amd import pararnn as pr

    case = s["case"]
    op = case["op"]
    if op == "step":
        new = pr.gated_step(s["u"], s["lam"], s["states"], slots=s["slots"], power=POWER)
        return new, s["states"]
    if op == "scan":
        return pr.gated_scan(s["u"], s["lam"], s["h0"], power=POWER, resets=s["resets"])
    if op == "scan_adjoint":
        return pr.gated_scan_adjoint(s["u"], s["lam"], s["h0"], s["h"], s["gh"], power=POWER,
                                     resets=s["resets"])
    if op == "block":
        return pr.block_norm(s["h"], s["x"], s["w_post"], s["w_pre"], gate=s["gate"], scale=SCALE,
                             eps=EPS)
    if op == "block_adjoint":
        return pr.block_norm_adjoint(s["h"], s["x"], s["w_post"], s["w_pre"], s["rstd"], s["gy"],
                                     s["gz"], gate=s["gate"], scale=SCALE)
    if op == "score":
        return pr.token_logprobs(s["logits"], s["tokens"], top=case["k"])
    return pr.token_logprobs_adjoint(s["logits"], s["tokens"], s["lse"], s["entropy"],
                                     g_logprob=s["g_logprob"], g_entropy=s["g_entropy"],
                                     g_lse=s["g_lse"])


def run(s):
    if own:
        return _own_run(s)
    op = s["case"]["op"]
    if op == "step":  # the states are updated in place, as a server keeps them
        new, states = _plain_step(s)
        s["states"].copy_(states)
        return new, s["states"]
    if op == "scan":
        return _plain_scan(s)
    if op == "scan_adjoint":
        return _plain_scan_adjoint(s)
    if op == "block":
        return _plain_block(s)
    if op == "block_adjoint":
        return _plain_block_adjoint(s)
    if op == "score":
        return _plain_score(s, s["case"]["k"])
    return _plain_score_adjoint(s)


# ------------------------------------------------------------------- exact ---

def _spans(a, b, start):
    """x_t = a_t x_{t-1} + b_t along the last axis, step by step; spans of the axis run side by
    side from zero, then each takes up the last value of the one before."""
    rows, T = a.shape[0], a.shape[1]
    span = max(1, int(math.sqrt(T)))
    count = -(-T // span)
    pad = count * span - T
    a = torch.nn.functional.pad(a, (0, pad)).view(rows, count, span)
    b = torch.nn.functional.pad(b, (0, pad)).view(rows, count, span)
    x, prod = torch.empty_like(b), torch.empty_like(a)
    value, product = torch.zeros_like(b[..., 0]), torch.ones_like(b[..., 0])
    for j in range(span):
        value = a[..., j] * value + b[..., j]
        product = product * a[..., j]
        x[..., j], prod[..., j] = value, product
    carry = start
    for c in range(count):
        x[:, c] += prod[:, c] * carry[:, None]
        carry = x[:, c, -1]
    return x.reshape(rows, -1)[:, :T]


def _exact_recurrence(s):
    u = [p.double() for p in s["u"]]
    soft = torch.nn.functional.softplus(s["lam"].double())
    soft = soft if u[0].dim() == 2 else soft[:, None]
    rate = 1.0 / (1.0 + torch.exp(-u[0]))
    l = -POWER * soft * rate
    gain = torch.sqrt(-torch.expm1(2.0 * l))
    return l, torch.exp(l), gain, 1.0 / (1.0 + torch.exp(-u[1])), u[2], rate


def exact(case, seed):
    op = case["op"]
    if _elements(case) > 300_000_000:
        return None
    s = prepare(case, seed)
    if op == "step":
        _, a, gain, i, x, _ = _exact_recurrence(s)
        states, new = s["states"].double(), torch.zeros(case["B"], case["D"], dtype=torch.float64, device="cuda")
        for row, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                new[row] = a[row] * states[slot] + gain[row] * i[row] * x[row]
                states[slot] = new[row]
        return new, states
    if op in ("scan", "scan_adjoint"):
        B, T, D = case["B"], case["T"], case["D"]
        l, a, gain, i, x, rate = _exact_recurrence(s)
        kept = a if s["resets"] is None else torch.where(s["resets"][:, None, :], 0.0, a)
        if op == "scan":
            b = gain * i * x
            del l, gain, i, x, rate
            h = _spans(kept.reshape(B * D, T), b.reshape(B * D, T), s["h0"].double().reshape(-1))
            h = h.reshape(B, D, T)
            return h, h[:, :, -1]
        gh = s["gh"].double()
        back = torch.zeros_like(kept)
        back[..., 1:] = kept[..., 1:].flip(-1)
        g = _spans(back.reshape(B * D, T), gh.flip(-1).reshape(B * D, T),
                   torch.zeros(B * D, dtype=torch.float64, device="cuda"))
        g = g.reshape(B, D, T).flip(-1)
        before = torch.empty_like(g)
        before[..., 0], before[..., 1:] = s["h0"].double(), s["h"].double()[..., :-1]
        d_l = g * (kept * before - torch.exp(2.0 * l) / gain * i * x)
        slope = torch.sigmoid(s["lam"].double())
        return dict(du=[d_l * l * (1.0 - rate), g * gain * x * i * (1.0 - i), g * gain * i],
                    dlam=-POWER * slope * (d_l * rate).sum(dim=(0, 2)), dh0=kept[..., 0] * g[..., 0])
    if op in ("block", "block_adjoint"):
        h = s["h"].double().transpose(1, 2).contiguous()
        g = s["gate"].double().transpose(1, 2).contiguous()
        x, wp, wn = s["x"].double(), s["w_post"].double(), s["w_pre"].double()
        act = g / (1.0 + torch.exp(-g))
        v = h * act
        r1 = 1.0 / torch.sqrt(v.square().mean(-1) + EPS)
        n1 = v * r1[..., None]
        y = x + SCALE * n1 * wp
        r2 = 1.0 / torch.sqrt(y.square().mean(-1) + EPS)
        n2 = y * r2[..., None]
        if op == "block":
            return y, n2 * wn, torch.stack([r1, r2])
        del y, x
        gz = s["gz"].double()
        inner = (gz * wn * n2).mean(-1, keepdim=True)
        gy = s["gy"].double() + r2[..., None] * (gz * wn - n2 * inner)
        inner = (SCALE * gy * wp * n1).mean(-1, keepdim=True)
        gv = r1[..., None] * (SCALE * gy * wp - n1 * inner)
        sig = act / g
        sig = torch.where(g == 0, 0.5, sig)
        return dict(dx=gy, dh=(gv * act).transpose(1, 2), dgate=(gv * h * (sig + act * (1.0 - sig))).transpose(1, 2),
                    dw_post=(SCALE * gy * n1).sum(dim=(0, 1)), dw_pre=(gz * n2).sum(dim=(0, 1)))
    logits, tokens = s["logits"], s["tokens"]
    N, V = logits.shape
    if op == "score_adjoint":
        grads = []
        for n in range(0, N, 256):  # a block of rows at a time
            x = logits[n:n + 256].double()
            t = tokens[n:n + 256]
            lse = torch.logsumexp(x, -1, keepdim=True)
            p = torch.nan_to_num(torch.exp(x - lse))
            logp = torch.where(p > 0, x - lse, 0.0)
            h = -(p * logp).sum(-1, keepdim=True)
            w = torch.where(t >= 0, s["g_logprob"][n:n + 256].double(), 0.0)[:, None]
            one = torch.zeros_like(x)
            rows = torch.nonzero((t >= 0) & ~torch.isneginf(lse[:, 0]))[:, 0]
            one[rows, t[rows]] = 1.0
            grad = w * (one - p) + s["g_lse"][n:n + 256].double()[:, None] * p
            grads.append(grad - s["g_entropy"][n:n + 256].double()[:, None] * p * (logp + h))
        return torch.cat(grads)
    out = dict(logprob=[], entropy=[], lse=[], top_index=[], top_logprob=[])
    for n in range(0, N, 256):
        x, t = logits[n:n + 256].double(), tokens[n:n + 256]
        lse = torch.logsumexp(x, -1, keepdim=True)
        empty = torch.isneginf(lse)
        logp = torch.where(empty, -math.inf, x - lse)
        out["lse"].append(lse[:, 0])
        out["logprob"].append(torch.where(t >= 0, logp.gather(1, t.clamp(min=0)[:, None])[:, 0], 0.0))
        p = torch.exp(logp)
        out["entropy"].append(-torch.where(p > 0, p * logp, 0.0).sum(-1))
        if case["k"]:
            best, at = torch.sort(x, dim=-1, descending=True, stable=True)
            best, at = best[:, :case["k"]], at[:, :case["k"]]
            out["top_logprob"].append(torch.where(torch.isneginf(best), -math.inf, best - lse))
            out["top_index"].append(torch.where(torch.isneginf(best), -1, at))
    return {name: torch.cat(parts) for name, parts in out.items() if parts}

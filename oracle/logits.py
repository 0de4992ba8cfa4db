"""Float64 oracle of the distillation from top tokens, forward and backward, and
of what is done to logits before sampling, row by row in numpy."""
import numpy as np

REST = 1e-6  # less is what rounding leaves of a full list


def _row(x, scale):
    """(log q of every token, lse); -inf where the row allows nothing."""
    z = scale * x
    if np.isnan(z).any() or np.isposinf(z).any():
        return np.full_like(z, np.nan), np.nan
    if np.isneginf(z).all():
        return np.full_like(z, -np.inf), -np.inf
    m = z.max()
    log_s = np.log(np.exp(z - m).sum())
    return z - m - log_s, m + log_s  # (next to a row of -1e38 the sum's logarithm is nothing)


def _sum_of(z):
    """log sum exp, also of numbers whose exponentials are 0 in float64."""
    m = z.max(initial=-np.inf)
    return m + np.log(np.exp(z - m).sum()) if np.isfinite(m) else m


def _teacher(index, logprob, tail):
    used = index >= 0
    p = np.where(used, np.exp(np.where(used, logprob, -np.inf)), 0.0)
    r = 1.0 - p.sum()
    return used, p, r if tail and r >= REST else 0.0


def distill_top(logits, index, logprob, tail=True, scale=1.0):
    """dict(loss, lse, log_rest)."""
    x = np.asarray(logits, np.float64)
    N, V = x.shape
    out = dict(loss=np.zeros(N), lse=np.zeros(N), log_rest=np.zeros(N))
    for n in range(N):
        logq, out["lse"][n] = _row(x[n], scale)
        used, p, r = _teacher(index[n], np.asarray(logprob[n], np.float64), tail)
        others = np.setdiff1d(np.arange(V), index[n][used])
        out["log_rest"][n] = rest = _sum_of(logq[others])
        if not used.any():
            continue
        if (index[n] >= V).any():
            out["loss"][n] = np.nan
            continue
        loss = sum(pe * (le - logq[j]) for j, pe, le in zip(index[n], p, logprob[n]) if j >= 0 and pe > 0)
        out["loss"][n] = loss + (r * (np.log(r) - rest) if r > 0 else 0.0)
    return out


def distill_top_adjoint(logits, index, logprob, g_loss, tail=True, scale=1.0):
    """dL/dlogits."""
    x = np.asarray(logits, np.float64)
    N, V = x.shape
    out = np.zeros_like(x)
    for n in range(N):
        logq, lse = _row(x[n], scale)
        used, p, r = _teacher(index[n], np.asarray(logprob[n], np.float64), tail)
        if not used.any() or np.isneginf(lse):
            continue
        q, P = np.exp(logq), p.sum()
        listed = np.zeros(V, bool)
        listed[index[n][used]] = True
        grad = q * (P + r)
        z = scale * x[n, ~listed]
        if r > 0 and not np.isneginf(z.max(initial=-np.inf)):  # (not from log q: next to a mask of -1e38 it is the mask)
            grad[~listed] -= r * np.exp(z - z.max() - _sum_of(z - z.max()))
        np.add.at(grad, index[n][used], -p[used])
        out[n] = g_loss[n] * scale * grad
    return out


def adjust_logits(logits, tokens=None, lengths=None, prompt=None, repetition=None, presence=None, frequency=None,
                  bias=None, allowed=None, allowed_rows=None):
    x = np.asarray(logits, np.float64).copy()
    N, V = x.shape
    for n in range(N):
        if tokens is not None:
            L = len(tokens[n]) if lengths is None else min(max(int(lengths[n]), 0), len(tokens[n]))
            first = 0 if prompt is None else int(prompt[n])
            seen, count = set(), {}
            for i in range(L):
                j = int(tokens[n][i])
                if 0 <= j < V:
                    seen.add(j)
                    if i >= first:
                        count[j] = count.get(j, 0) + 1
            rep = 1.0 if repetition is None else float(repetition[n])
            for j in seen:
                x[n, j] = x[n, j] / rep if x[n, j] > 0 else x[n, j] * rep
            for j, c in count.items():
                x[n, j] -= (0.0 if frequency is None else float(frequency[n])) * c
                x[n, j] -= 0.0 if presence is None else float(presence[n])
        if bias is not None:
            last = {int(j): float(b) for j, b in zip(bias[0][n], bias[1][n]) if 0 <= j < V}
            for j, b in last.items():
                x[n, j] += b
        if allowed is not None:
            r = n if allowed_rows is None else int(allowed_rows[n])
            if 0 <= r < len(allowed):
                words = np.asarray(allowed[r]).view(np.uint32)
                bits = (words[np.arange(V) // 32] >> (np.arange(V) % 32).astype(np.uint32)) & 1
                x[n, bits == 0] = -np.inf
    return x

"""torch.autograd bindings of the fused solve and its adjoint.

``gru(u, a, h0)`` and ``lstm(u, a, c0, h0)`` return the converged states and
record a backward that runs the reverse-time adjoint scan
(``pararnn_adjoint``) — gradients for the projections u, the diagonal weights
a and the initial states.  Both directions run in the HIP kernels; this
module only wires them into autograd (the pages' ParaRNN framework derives
the backward pass by autodiff in its PyTorch tier; here it is the adjoint of
the converged Newton solve, the transposed block-bidiagonal system of
"Параллельность RNN?" (forpes.ru), §1.3).

Two layouts: ``gru``/``lstm`` take one [B][D][T]-indexed tensor per gate
(any strides; channel-major is the fast layout), ``gru_time_major`` /
``lstm_time_major`` take the [B][T][G*D] tensor a ``torch.nn.Linear`` over
[B][T][I] inputs produces and return [B][T][D] states; its gate planes are
passed to the kernels as strided views (no transpose copy), and the
gradient for u comes back as one [B][T][G*D] tensor written by the adjoint.

``gated_scan``, ``delta_scan``, ``block_norm``, ``token_logprobs`` and
``distill_top`` are the differentiable forms of the operators of recurrent
language models.  They have first
derivatives: differentiating a gradient of theirs raises.  Their backward passes
can be captured in a HIP graph together with the forward ones; no eager graph of
the same leaves may be alive then, unless it was recorded on the stream of the
capture.  ``delta_scan`` and ``distill_top`` refuse a leaf that they are given where
such a graph is one of theirs, or was alive when they were last called on the leaf
outside of a capture; a leaf behind other operations is not seen.

Non-convergence is not an error in the solve; pass ``strict=True`` to raise
when a solve stops at the iteration cap without reaching the tolerance (this
reads the device info record, i.e. synchronises).
"""
import functools

import torch

from . import pararnn as pr


def _check(info_t, strict):
    if strict:
        info = pr.read_info(info_t)
        if not info["converged"]:
            raise RuntimeError(f"ParaRNN Newton solve did not converge: {info}")


def _grad_like(g, ref):
    return g if g.dtype == ref.dtype else g.to(ref.dtype)


def _strided_like(g, ref):
    """`g` with the strides of `ref` (the adjoint reads upstream gradients in
    the layout of the states)."""
    if g.stride() == ref.stride():
        return g
    out = torch.empty_strided(ref.shape, ref.stride(), dtype=g.dtype, device=g.device)
    out.copy_(g)
    return out


def _gate_planes(u, G):
    """Gate planes of a time-major [B][T][G*D] tensor as [B][D][T]-indexed
    views (no copy)."""
    if u.dim() != 3 or u.shape[2] % G != 0:
        raise ValueError(f"u must be [B][T][{G}*D]")
    D = u.shape[2] // G
    return [u[:, :, g * D:(g + 1) * D].transpose(1, 2) for g in range(G)]


def _time_major_adjoint(cell, u, a, s0, s, gs):
    """Adjoint for time-major tensors: u [B][T][G*D], s and gs [B][T][D]
    (gs entries may be None).  Returns (du [B][T][G*D], da, ds0 list)."""
    G = pr.N_GATES[pr.CELLS[cell]]
    B, T, GD = u.shape
    D = GD // G
    du = torch.empty((B, T, GD), dtype=torch.float32, device=u.device)
    da = torch.empty((G, D), dtype=torch.float32, device=u.device)
    ds0 = [torch.empty((B, D), dtype=torch.float32, device=u.device) for _ in s0]
    gsv = [None if g is None else g.contiguous().transpose(1, 2) for g in gs]
    pr.adjoint(cell, _gate_planes(u, G), a, s0, [x.transpose(1, 2) for x in s], gsv,
               out=dict(du=_gate_planes(du, G), da=da, ds0=ds0, lam=None))
    return du, da, ds0


class _GruSolve(torch.autograd.Function):
    @staticmethod
    def forward(ctx, uz, ur, uc, a, h0, tol, max_iters, strict):
        u = [uz, ur, uc]
        h, info_t = pr.solve_gru(u, a, h0, tol=tol, max_iters=max_iters, info=strict)
        _check(info_t, strict)
        ctx.save_for_backward(uz, ur, uc, a, h0, h)
        return h

    @staticmethod
    def backward(ctx, gh):
        uz, ur, uc, a, h0, h = ctx.saved_tensors
        out = pr.adjoint("gru", [uz, ur, uc], a, [h0], [h], [_strided_like(gh, h)])
        du = out["du"]
        return (_grad_like(du[0], uz), _grad_like(du[1], ur), _grad_like(du[2], uc),
                out["da"], out["ds0"][0], None, None, None)


class _LstmSolve(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ui, uf, ug, uo, a, c0, h0, tol, max_iters, strict):
        u = [ui, uf, ug, uo]
        (c, h), info_t = pr.solve_lstm(u, a, c0, h0, tol=tol, max_iters=max_iters, info=strict)
        _check(info_t, strict)
        ctx.save_for_backward(ui, uf, ug, uo, a, c0, h0, c, h)
        return c, h

    @staticmethod
    def backward(ctx, gc, gh):
        ui, uf, ug, uo, a, c0, h0, c, h = ctx.saved_tensors
        gs = [None if gc is None else _strided_like(gc, c),
              None if gh is None else _strided_like(gh, h)]
        out = pr.adjoint("lstm", [ui, uf, ug, uo], a, [c0, h0], [c, h], gs)
        du = out["du"]
        return (_grad_like(du[0], ui), _grad_like(du[1], uf), _grad_like(du[2], ug),
                _grad_like(du[3], uo), out["da"], out["ds0"][0], out["ds0"][1],
                None, None, None)


def gru(u, a, h0, *, tol=1e-6, max_iters=20, strict=False):
    """Differentiable ParaGRU solve.  u = (u_z, u_r, u_c) [B][D][T] device
    tensors; a [3][D]; h0 [B][D].  Returns h [B][D][T]."""
    uz, ur, uc = u
    return _GruSolve.apply(uz, ur, uc, a, h0, tol, max_iters, strict)


def lstm(u, a, c0, h0, *, tol=1e-6, max_iters=20, strict=False):
    """Differentiable ParaLSTM solve.  u = (u_i, u_f, u_g, u_o); a [4][D];
    c0, h0 [B][D].  Returns (c, h)."""
    ui, uf, ug, uo = u
    return _LstmSolve.apply(ui, uf, ug, uo, a, c0, h0, tol, max_iters, strict)


class _GruTimeMajor(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, a, h0, tol, max_iters, strict):
        B, T, _ = u.shape
        h = torch.empty((B, T, a.shape[1]), dtype=torch.float32, device=u.device)
        _, info_t = pr.solve_gru(_gate_planes(u, 3), a, h0, out=h.transpose(1, 2), tol=tol,
                                 max_iters=max_iters, info=strict)
        _check(info_t, strict)
        ctx.save_for_backward(u, a, h0, h)
        return h

    @staticmethod
    def backward(ctx, gh):
        u, a, h0, h = ctx.saved_tensors
        du, da, ds0 = _time_major_adjoint("gru", u, a, [h0], [h], [gh])
        return _grad_like(du, u), da, ds0[0], None, None, None


class _LstmTimeMajor(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, a, c0, h0, tol, max_iters, strict):
        B, T, _ = u.shape
        D = a.shape[1]
        c = torch.empty((B, T, D), dtype=torch.float32, device=u.device)
        h = torch.empty((B, T, D), dtype=torch.float32, device=u.device)
        _, info_t = pr.solve_lstm(_gate_planes(u, 4), a, c0, h0,
                                  out=[c.transpose(1, 2), h.transpose(1, 2)], tol=tol,
                                  max_iters=max_iters, info=strict)
        _check(info_t, strict)
        ctx.save_for_backward(u, a, c0, h0, c, h)
        return c, h

    @staticmethod
    def backward(ctx, gc, gh):
        u, a, c0, h0, c, h = ctx.saved_tensors
        du, da, ds0 = _time_major_adjoint("lstm", u, a, [c0, h0], [c, h], [gc, gh])
        return _grad_like(du, u), da, ds0[0], ds0[1], None, None, None


def gru_time_major(u, a, h0, *, tol=1e-6, max_iters=20, strict=False):
    """Differentiable ParaGRU solve on time-major tensors: u [B][T][3*D]
    (gate blocks z, r, c along the last dimension, float32 or bfloat16),
    a [3][D], h0 [B][D].  Returns h [B][T][D]."""
    return _GruTimeMajor.apply(u, a, h0, tol, max_iters, strict)


def lstm_time_major(u, a, c0, h0, *, tol=1e-6, max_iters=20, strict=False):
    """Differentiable ParaLSTM solve on time-major tensors: u [B][T][4*D]
    (gate blocks i, f, g, o), a [4][D], c0, h0 [B][D].  Returns (c, h), each
    [B][T][D]."""
    return _LstmTimeMajor.apply(u, a, c0, h0, tol, max_iters, strict)


class _NoSecondDerivative(torch.autograd.Function):
    """Its outputs, whose own derivative raises."""

    @staticmethod
    def forward(ctx, _, *tensors):
        return tuple(t.view_as(t) for t in tensors)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("trying to differentiate twice: the operators of recurrent language "
                           "models have first derivatives only")


def _once(backward):
    """A backward pass under ``create_graph`` gives gradients that cannot be
    differentiated, rather than constants.  (torch's ``once_differentiable``
    does so only where an incoming gradient depends on something: not for a
    sum of the outputs, though its gradient depends on the inputs.)"""
    @functools.wraps(backward)
    def wrapper(ctx, *grads):
        second = torch.is_grad_enabled()
        with torch.no_grad():
            out = backward(ctx, *grads)
        out = out if isinstance(out, tuple) else (out,)
        if not second:
            return out
        given = [i for i, t in enumerate(out) if t is not None]
        marked = _NoSecondDerivative.apply(torch.empty(0, requires_grad=True),
                                           *(out[i] for i in given))
        out = list(out)
        for i, t in zip(given, marked):
            out[i] = t
        return tuple(out)
    return wrapper


class _GatedScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ur, ui, ux, lam, h0, power, resets):
        h, h_last = pr.gated_scan([ur, ui, ux], lam, h0, power=power, resets=resets)
        ctx.save_for_backward(ur, ui, ux, lam, h0, resets, h)
        ctx.power = power
        ctx.set_materialize_grads(False)
        return h, h_last

    @staticmethod
    @_once
    def backward(ctx, gh, gh_last):
        ur, ui, ux, lam, h0, resets, h = ctx.saved_tensors
        out = pr.gated_scan_adjoint([ur, ui, ux], lam, h0, h,
                                    None if gh is None else _strided_like(gh, h),
                                    gh_last=None if gh_last is None else gh_last.contiguous(),
                                    power=ctx.power, resets=resets)
        return (*out["du"], out["dlam"], None if h0 is None else out["dh0"], None, None)


def gated_scan(u, lam, h0=None, *, power=8.0, resets=None):
    """Differentiable gated linear recurrence (``pararnn.gated_scan``): u =
    (u_r, u_i, u_x) [B][D][T], lam [D], h0 [B][D] or None.  Returns
    (h [B][D][T], h_last [B][D])."""
    ur, ui, ux = u
    return _GatedScan.apply(ur, ui, ux, lam, h0, power, resets)


_NOTE = "pararnn_stream"


def _stream_of(t):
    """(the current stream's handle on the tensor's device, whether it is being
    captured); None for a tensor that is not on a GPU."""
    if not t.is_cuda:
        return None
    stream = pr._raw_stream(t.device.index)
    return stream, bool(stream) and pr._capturing(t.device, stream)  # (the default stream, 0, cannot be captured)


def _record(function, *args):
    """``function.apply(*args)``, but no capture in which a leaf among the inputs
    is held by a graph that was recorded before it on another stream: the captured
    backward pass would have to wait for that stream, which ends the capture and
    with it the process.

    The node that collects a leaf's gradient belongs to the stream that it was made
    on, and lives as long as a graph holds it.  So the stream is noted on the nodes
    that the new graph holds.  A node that had no note before an eager call, and
    that another operator's graph holds, gets None: it may belong to any stream.
    (In a capture such a node is taken for the capture's own.)"""
    leaves = []
    if torch.is_grad_enabled():
        for t in args:
            if isinstance(t, torch.Tensor) and t.is_leaf and t.requires_grad:
                at = _stream_of(t)
                if at is not None:
                    leaves.append((t, *at))
    for t, stream, captured in leaves:
        # (a node that nobody holds is gone behind this statement, and its note with it)
        known = torch.autograd.graph.get_gradient_edge(t).node.metadata.setdefault(_NOTE, stream if captured else None)
        if captured and known != stream:
            raise RuntimeError("an input's gradient would be captured while an eager graph of it is alive: let "
                               "go of that graph's outputs first, or record it on the stream of the capture")
    out = function.apply(*args)
    if leaves:
        for node, _ in out[0].grad_fn.next_functions:
            if hasattr(node, "variable"):  # a leaf's
                node.metadata.setdefault(_NOTE, leaves[0][1])
    return out


class _DeltaScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, beta, log_decay, h0, scale, resets):
        if log_decay is not None and log_decay.shape == beta.shape and not pr._same_steps(log_decay, beta):
            beta, log_decay = beta.contiguous(), log_decay.contiguous()
        o, last = pr.delta_scan(q, k, v, beta, log_decay, h0, scale=scale, resets=resets)
        ctx.save_for_backward(q, k, v, beta, log_decay, h0, resets)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        return o, last

    @staticmethod
    @_once
    def backward(ctx, go, g_last):
        q, k, v, beta, log_decay, h0, resets = ctx.saved_tensors
        if go is not None:  # elements of their own, side by side as v's are
            strides = pr._like_steps(*v.shape, v)
            if go.stride() != strides:
                go = torch.empty_strided(go.shape, strides, dtype=go.dtype, device=go.device).copy_(go)
        out = pr.delta_scan_adjoint(q, k, v, beta, log_decay, h0, go,
                                    g_last=None if g_last is None else g_last.contiguous(), scale=ctx.scale,
                                    resets=resets)
        return (out["dq"], out["dk"], out["dv"], out["dbeta"], out["dlog_decay"], out["dh0"], None, None)


def delta_scan(q, k, v, beta, log_decay=None, h0=None, *, scale=None, resets=None):
    """Differentiable gated delta rule (``pararnn.delta_scan``): gradients for q,
    k, v, beta, log_decay and h0.  Returns (o [B][Hv][dv][T],
    last [B][Hv][dk][dv])."""
    return _record(_DeltaScan, q, k, v, beta, log_decay, h0, scale, resets)


class _BlockNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, gate, x, w_post, w_pre, scale, eps, z_dtype):
        y, z, rstd = pr.block_norm(h, x, w_post, w_pre, gate=gate, scale=scale, eps=eps,
                                   z_dtype=z_dtype)
        ctx.save_for_backward(h, gate, x, w_post, w_pre, rstd)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        return x.view_as(x) if h is None else y, z

    @staticmethod
    @_once
    def backward(ctx, gy, gz):
        h, gate, x, w_post, w_pre, rstd = ctx.saved_tensors
        out = pr.block_norm_adjoint(h, x, w_post, w_pre, rstd,
                                    None if gy is None else _strided_like(gy, x),
                                    None if gz is None else gz.contiguous(), gate=gate,
                                    scale=ctx.scale)
        return (out["dh"], out["dgate"], out["dx"], out["dw_post"], out["dw_pre"], None, None,
                None)


def block_norm(h, x, w_post, w_pre, *, gate=None, scale=1.0, eps=1e-6, z_dtype=torch.bfloat16):
    """Differentiable block boundary (``pararnn.block_norm``).  Returns (y, z)."""
    return _BlockNorm.apply(h, gate, x, w_post, w_pre, scale, eps, z_dtype)


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, top, scale):
        out = pr.token_logprobs(logits, tokens, top=top, scale=scale)
        ctx.save_for_backward(logits, tokens, out["lse"], out["entropy"])
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        tops = (out["top_index"], out["top_logprob"]) if top else ()
        ctx.mark_non_differentiable(*tops)
        return (out["logprob"], out["entropy"], out["lse"]) + tops

    @staticmethod
    @_once
    def backward(ctx, g_logprob, g_entropy, g_lse, *_):
        logits, tokens, lse, entropy = ctx.saved_tensors
        g = [None if x is None else x.contiguous() for x in (g_logprob, g_entropy, g_lse)]
        return (pr.token_logprobs_adjoint(logits, tokens, lse, entropy, g_logprob=g[0],
                                          g_entropy=g[1], g_lse=g[2], scale=ctx.scale),
                None, None, None)


def token_logprobs(logits, tokens, *, top=0, scale=1.0):
    """Differentiable token scores (``pararnn.token_logprobs``): gradients for
    the logits from logprob, entropy and lse; the alternatives carry none."""
    out = _TokenLogprobs.apply(logits, tokens, int(top), scale)
    names = ("logprob", "entropy", "lse", "top_index", "top_logprob")
    return dict(zip(names, out))


class _DistillTop(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, top_index, top_logprob, tail, scale):
        out = pr.distill_top(logits, top_index, top_logprob, tail=tail, scale=scale)
        ctx.save_for_backward(logits, top_index, top_logprob, out["lse"], out["log_rest"])
        ctx.tail, ctx.scale = tail, scale
        ctx.mark_non_differentiable(out["lse"], out["log_rest"])
        return out["loss"], out["lse"], out["log_rest"]

    @staticmethod
    @_once
    def backward(ctx, g_loss, *_):
        logits, top_index, top_logprob, lse, log_rest = ctx.saved_tensors
        return (pr.distill_top_adjoint(logits, top_index, top_logprob, lse, log_rest, g_loss.contiguous(),
                                       tail=ctx.tail, scale=ctx.scale), None, None, None, None)


def distill_top(logits, top_index, top_logprob, *, tail=True, scale=1.0):
    """Differentiable distillation loss (``pararnn.distill_top``): the gradient
    of the loss for the student's logits; lse and log_rest carry none, and the
    teacher's list is taken as given."""
    loss, lse, log_rest = _record(_DistillTop, logits, top_index, top_logprob, tail, scale)
    return dict(loss=loss, lse=lse, log_rest=log_rest)

"""What the gated delta rule, the distillation and the logits before sampling
refuse, on the CPU: the C ABI checks its arguments before any HIP call, and the
binding names the first thing that is wrong before it calls the library."""
import ctypes
import math

import pytest
import torch

from nonlinear_rnn_amd import pararnn as pr

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = 256  # stands for a device pointer; nothing may be read through it
NULL = None


def dense(*size):
    out = [1]
    for n in reversed(size[1:]):
        out.insert(0, out[0] * n)
    return out


def shape(B=2, T=5, Hk=2, Hv=4, dk=3, dv=6, **strides):
    four, three = ctypes.c_int64 * 4, ctypes.c_int64 * 3
    s = dict(q=dense(B, Hk, dk, T), k=dense(B, Hk, dk, T), v=dense(B, Hv, dv, T), o=dense(B, Hv, dv, T),
             gate=dense(B, Hv, T)) | strides
    return pr.DeltaShape(B, T, Hk, Hv, dk, dv, four(*s["q"]), four(*s["k"]), four(*s["v"]), four(*s["o"]),
                         three(*s["gate"]))


def grads(**kw):
    """Of shape()'s sizes."""
    four = ctypes.c_int64 * 4
    g = dict(dq=P, dk=P, dv=P, q=dense(2, 2, 3, 5), k=dense(2, 2, 3, 5), v=dense(2, 4, 6, 5), dbeta=P, dlog=P) | kw
    return pr.DeltaGrads(g["dq"], g["dk"], g["dv"], four(*g["q"]), four(*g["k"]), four(*g["v"]), g["dbeta"],
                         g["dlog"], NULL)


SHAPES = [
    (dict(sh=NULL), INVALID), (dict(sh=shape(B=-1)), INVALID), (dict(sh=shape(T=-1)), INVALID),
    (dict(sh=shape(Hk=-1)), INVALID), (dict(sh=shape(Hv=5)), INVALID), (dict(sh=shape(Hv=0)), INVALID),
    (dict(sh=shape(Hk=0)), INVALID), (dict(sh=shape(dk=0)), INVALID), (dict(sh=shape(dv=0)), INVALID),
    (dict(sh=shape(q=[30, 15, 5, -1])), INVALID), (dict(sh=shape(v=[120, 30, -5, 1])), INVALID),
    (dict(sh=shape(gate=[20, 5, -1])), INVALID), (dict(sh=shape(k=[2 ** 62, 15, 5, 1])), INVALID),
    (dict(dt=2), UNSUPPORTED), (dict(sh=shape(dk=257)), UNSUPPORTED), (dict(sh=shape(dv=2 ** 20 + 1)), UNSUPPORTED),
    (dict(sh=shape(B=2 ** 23, T=1)), UNSUPPORTED), (dict(sh=shape(T=2 ** 30)), UNSUPPORTED),
    (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID),
    (dict(q=NULL), INVALID), (dict(k=NULL), INVALID), (dict(v=NULL), INVALID), (dict(beta=NULL), INVALID),
    (dict(ws=NULL), WORKSPACE), (dict(n=64), WORKSPACE), (dict(ws=P + 4), WORKSPACE)]


def common(kw):
    a = dict(sh=shape(), q=P, k=P, v=P, dt=0, beta=P, log_decay=P, scale=1.0, o=P, go=P, g=grads(), ws=P,
             n=1 << 40) | kw
    ref = None if a["sh"] is None else ctypes.byref(a["sh"])
    return a, (ref, a["q"], a["k"], a["v"], a["dt"], a["beta"], a["log_decay"], NULL, NULL, a["scale"])


@pytest.mark.parametrize("kw,status", SHAPES + [
    (dict(sh=shape(o=[120, 30, 4, 1])), INVALID), (dict(sh=shape(o=[120, 30, 0, 1])), INVALID),
    (dict(o=NULL), INVALID)])
def test_delta_scan(kw, status):
    a, head = common(kw)
    assert pr.load().pararnn_delta_scan(*head, a["o"], NULL, a["ws"], a["n"], NULL) == status


@pytest.mark.parametrize("kw,status", SHAPES + [
    (dict(g=NULL), INVALID), (dict(g=grads(dq=NULL)), INVALID), (dict(g=grads(dk=NULL)), INVALID),
    (dict(g=grads(dv=NULL)), INVALID), (dict(g=grads(dbeta=NULL)), INVALID), (dict(g=grads(dlog=NULL)), INVALID),
    (dict(g=grads(q=[30, 15, 0, 1])), INVALID), (dict(g=grads(v=[120, 30, 4, 1])), INVALID)])
def test_delta_scan_adjoint(kw, status):
    a, head = common(kw)
    g = None if a["g"] is None else ctypes.byref(a["g"])
    assert pr.load().pararnn_delta_scan_adjoint(*head, a["go"], NULL, g, a["ws"], a["n"], NULL) == status


@pytest.mark.parametrize("kw,status", [
    (dict(sh=NULL), INVALID), (dict(sh=shape(T=2)), INVALID), (dict(sh=shape(T=1, Hv=3)), INVALID),
    (dict(pool=-1), INVALID), (dict(q=NULL), INVALID), (dict(v=NULL), INVALID), (dict(beta=NULL), INVALID),
    (dict(states=NULL), INVALID), (dict(o=NULL), INVALID), (dict(scale=math.nan), INVALID), (dict(dt=4), UNSUPPORTED),
    (dict(sh=shape(T=1, dk=300)), UNSUPPORTED), (dict(sh=shape(T=1, B=2 ** 30)), UNSUPPORTED),
    (dict(sh=shape(T=1, o=[24, 3, 1, 1])), INVALID), (dict(sh=shape(T=1, B=0)), OK)])
def test_delta_step(kw, status):
    a = dict(sh=shape(T=1), q=P, k=P, v=P, dt=0, beta=P, states=P, pool=4, scale=1.0, o=P) | kw
    ref = None if a["sh"] is None else ctypes.byref(a["sh"])
    assert pr.load().pararnn_delta_step(ref, a["q"], a["k"], a["v"], a["dt"], a["beta"], NULL, NULL, a["states"],
                                        a["pool"], a["scale"], a["o"], NULL) == status


DISTILL = [
    (dict(N=-1), INVALID), (dict(V=-1), INVALID), (dict(stride=99), INVALID), (dict(stride=2 ** 62), INVALID),
    (dict(dt=3), UNSUPPORTED), (dict(top=-1), INVALID), (dict(top=pr.DISTILL_MAX + 1), UNSUPPORTED),
    (dict(scale=0.0), INVALID), (dict(scale=math.inf), INVALID), (dict(N=2 ** 24), UNSUPPORTED), (dict(x=NULL), INVALID),
    (dict(index=NULL), INVALID), (dict(logprob=NULL), INVALID), (dict(lse=NULL), INVALID), (dict(rest=NULL), INVALID),
    (dict(N=0), OK)]


@pytest.mark.parametrize("kw,status", DISTILL + [
    (dict(loss=NULL), INVALID), (dict(V=200000, stride=200000), WORKSPACE)])
def test_distill_top(kw, status):
    a = dict(N=3, V=100, x=P, dt=0, stride=100, index=P, logprob=P, top=2, scale=1.0, loss=P, lse=P, rest=P) | kw
    got = pr.load().pararnn_distill_top(a["N"], a["V"], a["x"], a["dt"], a["stride"], a["index"], a["logprob"],
                                        a["top"], 1, a["scale"], a["loss"], a["lse"], a["rest"], NULL, 0, NULL)
    assert got == status


@pytest.mark.parametrize("kw,status", DISTILL + [
    (dict(g=NULL), INVALID), (dict(dx=NULL), INVALID), (dict(dstride=50), INVALID), (dict(dx=P, dstride=101), INVALID),
    (dict(V=0), OK)])
def test_distill_top_adjoint(kw, status):
    a = dict(N=3, V=100, x=P, dt=0, stride=100, index=P, logprob=P, top=2, scale=1.0, lse=P, rest=P, g=P, dx=2 * P,
             dstride=100) | kw
    got = pr.load().pararnn_distill_top_adjoint(a["N"], a["V"], a["x"], a["dt"], a["stride"], a["index"],
                                                a["logprob"], a["top"], 1, a["scale"], a["lse"], a["rest"], a["g"],
                                                a["dx"], a["dstride"], NULL)
    assert got == status


@pytest.mark.parametrize("kw,status", [
    (dict(how=NULL), INVALID), (dict(N=-1), INVALID), (dict(V=-3), INVALID), (dict(stride=99), INVALID),
    (dict(out_stride=99), INVALID), (dict(dt=9), UNSUPPORTED), (dict(N=2 ** 24), UNSUPPORTED), (dict(x=NULL), INVALID),
    (dict(out=NULL), INVALID), (dict(out=P, out_stride=200), INVALID), (dict(length=4), INVALID),
    (dict(length=-1), INVALID), (dict(tokens=P, length=4, token_stride=-4), INVALID), (dict(biases=2), INVALID),
    (dict(biases=-2), INVALID), (dict(biases=2, bias_index=P), INVALID), (dict(allowed=P, allowed_stride=3), INVALID),
    (dict(allowed=P, allowed_stride=4, allowed_count=2), INVALID), (dict(length=2 ** 31), UNSUPPORTED),
    (dict(N=0), OK), (dict(V=0), OK)])
def test_adjust_logits(kw, status):
    a = dict(N=3, V=100, x=P, dt=0, stride=100, out=2 * P, out_stride=100, how=0, tokens=NULL, token_stride=4, length=0,
             bias_index=NULL, bias_value=NULL, biases=0, allowed=NULL, allowed_stride=0, allowed_count=0) | kw
    how = pr.Adjust(a["tokens"], a["token_stride"], a["length"], NULL, NULL, NULL, NULL, NULL, a["bias_index"],
                    a["bias_value"], a["biases"], a["allowed"], a["allowed_stride"], a["allowed_count"], NULL)
    got = pr.load().pararnn_adjust_logits(a["N"], a["V"], a["x"], a["dt"], a["stride"],
                                          None if a["how"] is None else ctypes.byref(how), a["out"], a["out_stride"],
                                          NULL)
    assert got == status


def test_workspace_sizes():
    size = pr.load().pararnn_delta_workspace_bytes
    few, many = shape(1, 65536, 4, 4, 64, 64), shape(64, 1024, 4, 4, 64, 64)
    # an inverse of each chunk of 32 steps; of few heads the segments' maps as well
    assert size(ctypes.byref(many), 0, 0) == 64 * 4 * 32 * 32 * 32 * 4
    assert size(ctypes.byref(few), 0, 0) > 4 * 2048 * 32 * 32 * 4
    # the states before and behind each chunk
    assert size(ctypes.byref(many), 0, 1) > 2 * 64 * 4 * 32 * 64 * 64 * 4
    assert size(ctypes.byref(shape(B=-1)), 0, 0) == 0 and size(ctypes.byref(shape(T=0)), 0, 1) == 0
    assert pr.load().pararnn_distill_workspace_bytes(4096, 50003) == 0
    assert pr.load().pararnn_distill_workspace_bytes(2, 131072) > 0


# The binding: tensors on the CPU pass every check but the last one.

def heads(B=2, Hk=1, Hv=2, dk=3, dv=4, T=5, dtype=torch.float32, **kw):
    z = dict(q=torch.zeros((B, Hk, dk, T), dtype=dtype), k=torch.zeros((B, Hk, dk, T), dtype=dtype),
             v=torch.zeros((B, Hv, dv, T), dtype=dtype), beta=torch.zeros(B, Hv, T)) | kw
    return z


def step(**kw):
    z = dict(q=torch.zeros(2, 1, 3), k=torch.zeros(2, 1, 3), v=torch.zeros(2, 2, 4), beta=torch.zeros(2, 2),
             log_decay=None, states=torch.zeros(3, 2, 3, 4)) | kw
    return pr.delta_step(**z)


def adjoint(go=None, **kw):
    z = heads() | kw
    return pr.delta_scan_adjoint(z["q"], z["k"], z["v"], z["beta"], None, None, go, **{n: z[n] for n in z if n == "g_last"})


def teacher(N=2, k=3):
    return torch.zeros((N, k), dtype=torch.int64), torch.zeros(N, k)


X = torch.zeros(2, 40)


@pytest.mark.parametrize("call,message", [
    (lambda: pr.delta_scan(**heads(dtype=torch.float16)), "float32 or bfloat16"),
    (lambda: pr.delta_scan(**heads(v=None)), "v"), (lambda: pr.delta_scan(**heads(q=torch.zeros(2, 3, 5))), "q"),
    (lambda: pr.delta_scan(**heads(k=torch.zeros(2, 1, 2, 5))), "k"),
    (lambda: pr.delta_scan(**heads(k=torch.zeros(2, 1, 3, 5).bfloat16())), "dtype"),
    (lambda: pr.delta_scan(**heads(v=torch.zeros(2, 2, 4, 6))), "batch and time"),
    (lambda: pr.delta_scan(**heads(Hk=2, Hv=3)), "multiple"), (lambda: pr.delta_scan(**heads(dk=257)), "256"),
    (lambda: pr.delta_scan(**heads(beta=torch.zeros(2, 2, 4))), "beta"),
    (lambda: pr.delta_scan(**heads(log_decay=torch.zeros(2, 2, 5).bfloat16())), "log_decay"),
    (lambda: pr.delta_scan(**heads(log_decay=torch.zeros(2, 5, 2).transpose(1, 2))), "strides"),
    (lambda: pr.delta_scan(**heads(h0=torch.zeros(2, 2, 4, 3))), "h0"),
    (lambda: pr.delta_scan(**heads(resets=torch.zeros(2, 5))), "resets"),
    (lambda: pr.delta_scan(**heads(out=torch.zeros(2, 2, 4, 4))), "out"), (lambda: pr.delta_scan(**heads()), "GPU"),
    (lambda: adjoint(go=torch.zeros(2, 2, 4, 4)), "go"), (lambda: adjoint(g_last=torch.zeros(2, 2, 3)), "g_last"),
    (lambda: adjoint(), "GPU"),
    (lambda: step(q=torch.zeros(2, 3)), "q"), (lambda: step(beta=torch.zeros(2, 3)), "beta"),
    (lambda: step(states=torch.zeros(3, 2, 4, 3)), "states"), (lambda: step(states=torch.zeros(1, 2, 3, 4)), "slots"),
    (lambda: step(slots=torch.zeros(2)), "int32"), (lambda: step(out=torch.zeros(2, 2, 3)), "out"),
    (lambda: step(), "GPU"),
    (lambda: pr.distill_top(X.double(), *teacher()), "logits"), (lambda: pr.distill_top(X.t(), *teacher(40)), "contiguous"),
    (lambda: pr.distill_top(X, teacher()[0].int(), teacher()[1]), "top_index"),
    (lambda: pr.distill_top(X, *teacher(3)), "top_index"), (lambda: pr.distill_top(X, *teacher(2, 1025)), "1024"),
    (lambda: pr.distill_top(X, teacher()[0], torch.zeros(2, 2)), "top_logprob"),
    (lambda: pr.distill_top(X, *teacher()), "GPU"),
    (lambda: pr.distill_top_adjoint(X, *teacher(), torch.zeros(2), torch.zeros(3), torch.zeros(2)), "log_rest"),
    (lambda: pr.distill_top_adjoint(X, *teacher(), torch.zeros(2), torch.zeros(2), torch.zeros(2),
                                    out=X.bfloat16()), "out"),
    (lambda: pr.adjust_logits(X.half()), "logits"), (lambda: pr.adjust_logits(X, tokens=torch.zeros(2, 3)), "tokens"),
    (lambda: pr.adjust_logits(X, repetition=torch.ones(2)), "needs tokens"),
    (lambda: pr.adjust_logits(X, tokens=torch.zeros(2, 3).long(), lengths=torch.zeros(2).long()), "lengths"),
    (lambda: pr.adjust_logits(X, tokens=torch.zeros(2, 3).long(), presence=torch.zeros(3)), "presence"),
    (lambda: pr.adjust_logits(X, bias=(torch.zeros(2, 3).long(), torch.zeros(2, 2))), "bias"),
    (lambda: pr.adjust_logits(X, allowed=torch.zeros(2, 1).int()), "allowed"),
    (lambda: pr.adjust_logits(X, allowed=torch.zeros(1, 2).int()), "allowed_rows"),
    (lambda: pr.adjust_logits(X, allowed=torch.zeros(2).int().expand(2, 2)), "overlap"),
    (lambda: pr.adjust_logits(X, allowed_rows=torch.zeros(2).int()), "needs allowed"),
    (lambda: pr.adjust_logits(X, allowed=torch.zeros(1, 2).int(), allowed_rows=torch.zeros(2)), "allowed_rows"),
    (lambda: pr.adjust_logits(X, out=torch.zeros(2, 39)), "out"), (lambda: pr.adjust_logits(X), "GPU"),
])
def test_binding(call, message):
    for _ in range(2):  # the second time as well: a refusal is not remembered as a plan
        with pytest.raises(ValueError, match=message):
            call()

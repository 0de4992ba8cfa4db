"""What the operators of language models refuse, on the CPU: the C ABI checks
its arguments before any HIP call, and the binding names the first thing that
is wrong before it calls the library."""
import ctypes
import math

import pytest
import torch

from nonlinear_rnn_amd import pararnn as pr

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = 256  # stands for a device pointer; nothing may be read through it
NULL = None


def ptrs(*values):
    return (ctypes.c_void_p * len(values))(*values)


def shape(B=2, T=5, D=3, u=None, s=None):
    return ctypes.byref(pr.make_shape(B, T, D, u, s))


def scan(sh=None, u=ptrs(P, P, P), dt=0, lam=P, power=8.0, h=P, ws=NULL, ws_bytes=0):
    return pr.load().pararnn_gated_scan(sh or shape(), u, dt, lam, power, NULL, NULL, h, NULL, ws,
                                        ws_bytes, NULL)


def scan_adjoint(sh=None, u=ptrs(P, P, P), dt=0, lam=P, h=P, du=ptrs(P, P, P), dlam=P, ws=P,
                 ws_bytes=1 << 30):
    return pr.load().pararnn_gated_scan_adjoint(sh or shape(), u, dt, lam, 8.0, NULL, NULL, h, NULL,
                                                NULL, du, dlam, NULL, ws, ws_bytes, NULL)


@pytest.mark.parametrize("kw,status", [
    (dict(sh=shape(B=-1)), INVALID), (dict(sh=shape(u=(0, 5, 1))), INVALID),
    (dict(sh=shape(s=(15, 4, 1))), INVALID), (dict(sh=shape(u=(15, 5, -1))), INVALID),
    (dict(u=NULL), INVALID), (dict(u=ptrs(P, NULL, P)), INVALID), (dict(lam=NULL), INVALID),
    (dict(h=NULL), INVALID), (dict(dt=2), UNSUPPORTED), (dict(power=0.0), INVALID),
    (dict(power=-1.0), INVALID), (dict(power=math.nan), INVALID), (dict(power=math.inf), INVALID),
    (dict(sh=shape(B=2 ** 20, D=2 ** 20, T=1, u=(2 ** 20, 1, 1), s=(2 ** 20, 1, 1))), UNSUPPORTED),
    (dict(sh=shape(1, 100000, 2)), WORKSPACE), (dict(sh=shape(1, 100000, 2), ws=P, ws_bytes=8), WORKSPACE),
    (dict(sh=shape(1, 100000, 2), ws=P + 4, ws_bytes=1 << 30), WORKSPACE)])
def test_gated_scan(kw, status):
    assert scan(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(h=NULL), INVALID), (dict(du=NULL), INVALID), (dict(du=ptrs(P, P, NULL)), INVALID),
    (dict(dlam=NULL), INVALID), (dict(lam=NULL), INVALID), (dict(ws=NULL), WORKSPACE),
    (dict(ws_bytes=1), WORKSPACE)])
def test_gated_scan_adjoint(kw, status):
    assert scan_adjoint(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), INVALID), (dict(pool=-1), INVALID), (dict(stride=2), INVALID), (dict(dt=7), UNSUPPORTED),
    (dict(power=math.nan), INVALID), (dict(u=ptrs(P, P, NULL)), INVALID), (dict(states=NULL), INVALID),
    (dict(out=NULL), INVALID), (dict(lam=NULL), INVALID), (dict(B=0), OK), (dict(B=2 ** 31), UNSUPPORTED)])
def test_gated_step(kw, status):
    a = dict(B=2, D=3, u=ptrs(P, P, P), dt=0, stride=3, lam=P, power=8.0, states=P, pool=4, out=P) | kw
    got = pr.load().pararnn_gated_step(a["B"], a["D"], a["u"], a["dt"], a["stride"], a["lam"], a["power"],
                                       NULL, a["states"], a["pool"], a["out"], NULL)
    assert got == status


def block_shape(B=2, T=5, D=3, **kw):
    s = dict(B=B, T=T, D=D, h_stride_b=D * T, h_stride_d=T, h_stride_t=1, g_stride_b=D * T, g_stride_d=T,
             g_stride_t=1, x_stride_b=D * T, x_stride_t=D, z_stride_b=D * T, z_stride_t=D) | kw
    return ctypes.byref(pr.BlockShape(**s))


@pytest.mark.parametrize("kw,status", [
    (dict(sh=block_shape(T=-1)), INVALID), (dict(sh=block_shape(h_stride_d=4)), INVALID),
    (dict(sh=block_shape(x_stride_t=2)), INVALID), (dict(sh=block_shape(z_stride_b=1)), INVALID),
    (dict(x=NULL), INVALID), (dict(wn=NULL), INVALID), (dict(wp=NULL), INVALID), (dict(z=NULL), INVALID),
    (dict(y=NULL), INVALID), (dict(h=NULL), INVALID), (dict(eps=0.0), INVALID), (dict(eps=math.nan), INVALID),
    (dict(scale=math.inf), INVALID), (dict(xdt=3), UNSUPPORTED), (dict(gdt=-1), UNSUPPORTED),
    (dict(zdt=9), UNSUPPORTED), (dict(sh=block_shape(B=0)), OK), (dict(sh=block_shape(D=0)), OK)])
def test_block_norm(kw, status):
    a = dict(sh=block_shape(), h=P, gate=P, gdt=0, x=P, xdt=0, wp=P, wn=P, scale=1.0, eps=1e-6, y=P, z=P,
             zdt=1) | kw
    got = pr.load().pararnn_block_norm(a["sh"], a["h"], a["gate"], a["gdt"], a["x"], a["xdt"], a["wp"],
                                       a["wn"], a["scale"], a["eps"], a["y"], a["z"], a["zdt"], NULL, NULL)
    assert got == status


@pytest.mark.parametrize("kw,status", [
    (dict(rstd=NULL), INVALID), (dict(dx=NULL), INVALID), (dict(dh=NULL), INVALID), (dict(dg=NULL), INVALID),
    (dict(dwp=NULL), INVALID), (dict(dwn=NULL), INVALID), (dict(ws=NULL), WORKSPACE), (dict(n=4), WORKSPACE),
    (dict(scale=math.nan), INVALID)])
def test_block_norm_adjoint(kw, status):
    a = dict(sh=block_shape(), rstd=P, dh=P, dg=P, dx=P, dwp=P, dwn=P, ws=P, n=1 << 30, scale=1.0) | kw
    got = pr.load().pararnn_block_norm_adjoint(a["sh"], P, P, 0, P, 0, P, P, a["scale"], a["rstd"], NULL, NULL,
                                               0, a["dh"], a["dg"], a["dx"], a["dwp"], a["dwn"], a["ws"],
                                               a["n"], NULL)
    assert got == status


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), INVALID), (dict(stride=99), INVALID), (dict(stride=2 ** 62), INVALID), (dict(x=NULL), INVALID),
    (dict(tokens=NULL), INVALID), (dict(logprob=NULL), INVALID), (dict(top=1, index=NULL), INVALID),
    (dict(top=-1), INVALID), (dict(top=pr.TOP_MAX + 1), UNSUPPORTED), (dict(scale=0.0), INVALID),
    (dict(scale=math.nan), INVALID), (dict(dt=5), UNSUPPORTED), (dict(N=2 ** 24), UNSUPPORTED),
    (dict(N=0), OK), (dict(V=200000, stride=200000), WORKSPACE)])
def test_token_logprobs(kw, status):
    a = dict(N=3, V=100, x=P, dt=0, stride=100, tokens=P, top=0, scale=1.0, logprob=P, index=P) | kw
    got = pr.load().pararnn_token_logprobs(a["N"], a["V"], a["x"], a["dt"], a["stride"], a["tokens"], a["top"],
                                           a["scale"], a["logprob"], NULL, NULL, a["index"], P, NULL, 0, NULL)
    assert got == status


@pytest.mark.parametrize("kw,status", [
    (dict(lse=NULL), INVALID), (dict(dx=NULL), INVALID), (dict(ge=P, entropy=NULL), INVALID),
    (dict(dstride=50), INVALID), (dict(dx=P, x=P, dstride=101), INVALID), (dict(scale=-2.0), INVALID)])
def test_token_logprobs_adjoint(kw, status):
    a = dict(x=P, lse=P, entropy=P, ge=NULL, dx=2 * P, dstride=100, scale=1.0) | kw
    got = pr.load().pararnn_token_logprobs_adjoint(3, 100, a["x"], 0, 100, P, a["scale"], a["lse"], a["entropy"],
                                                   NULL, a["ge"], NULL, a["dx"], a["dstride"], NULL)
    assert got == status


def test_workspace_sizes():
    lib = pr.load()
    assert lib.pararnn_gated_workspace_bytes(shape(8, 4096, 1024), 0) == 0
    assert lib.pararnn_gated_workspace_bytes(shape(1, 262144, 64), 0) > 0
    assert lib.pararnn_gated_workspace_bytes(shape(8, 4096, 1024), 1) >= 8 * 1024 * 4
    assert lib.pararnn_gated_workspace_bytes(shape(B=-1), 1) == 0
    assert lib.pararnn_block_workspace_bytes(block_shape(8, 4096, 1024)) >= 2 * 1024 * 4
    assert lib.pararnn_logprobs_workspace_bytes(4096, 50003, 8) == 0
    assert lib.pararnn_logprobs_workspace_bytes(2, 131072, 8) > 0
    assert lib.pararnn_logprobs_workspace_bytes(2, 131072, pr.TOP_MAX + 1) == 0


# The binding: tensors on the CPU pass every check but the last one.

def planes(B=2, D=3, T=5, n=3, dtype=torch.float32):
    return [torch.zeros((B, D, T), dtype=dtype) for _ in range(n)]


@pytest.mark.parametrize("call,message", [
    (lambda: pr.gated_scan(planes(n=2), torch.zeros(3)), "expected 3"),
    (lambda: pr.gated_scan(planes(dtype=torch.float16), torch.zeros(3)), "float32 or bfloat16"),
    (lambda: pr.gated_scan(planes(), torch.zeros(4)), "lam"),
    (lambda: pr.gated_scan(planes(), torch.zeros(3), torch.zeros(2, 2)), "h0"),
    (lambda: pr.gated_scan(planes(), torch.zeros(3), resets=torch.zeros(2, 5)), "resets"),
    (lambda: pr.gated_scan(planes(), torch.zeros(3), resets=torch.zeros(5, 2, dtype=torch.bool)), "resets"),
    (lambda: pr.gated_scan(planes(2), torch.zeros(3), out=torch.zeros(2, 3, 4)), "out"),
    (lambda: pr.gated_scan(planes(), torch.zeros(3)), "GPU"),
    (lambda: pr.gated_scan([1, 2, 3], torch.zeros(3)), "u"),
    (lambda: pr.gated_scan_adjoint(planes(), torch.zeros(3), None, torch.zeros(2, 3, 5), torch.zeros(2, 5, 3).transpose(1, 2)), "strides"),
    (lambda: pr.gated_scan_adjoint(planes(), torch.zeros(3), None, None, None), "h"),
    (lambda: pr.gated_scan_adjoint(planes(), torch.zeros(3), None, torch.zeros(2, 3, 5), None, gh_last=torch.zeros(3, 2)), "gh_last"),
    (lambda: pr.gated_step([torch.zeros(2, 3)] * 2, torch.zeros(3), torch.zeros(4, 3)), "3 gate"),
    (lambda: pr.gated_step([torch.zeros(2, 3)] * 3, torch.zeros(3), torch.zeros(1, 3)), "slots"),
    (lambda: pr.gated_step([torch.zeros(2, 3)] * 3, torch.zeros(3), torch.zeros(4, 2)), "states"),
    (lambda: pr.gated_step([torch.zeros(2, 3)] * 3, torch.zeros(3), torch.zeros(4, 3), slots=torch.zeros(2)), "int32"),
    (lambda: pr.gated_step([torch.zeros(3, 2).t()] * 3, torch.zeros(3), torch.zeros(4, 3)), "contiguous"),
    (lambda: pr.block_norm(torch.zeros(2, 5, 3), torch.zeros(2, 5, 3), torch.ones(3), torch.ones(3)), "h"),
    (lambda: pr.block_norm(None, torch.zeros(2, 5, 3), None, torch.ones(3), gate=torch.zeros(2, 3, 5)), "gate"),
    (lambda: pr.block_norm(None, torch.zeros(2, 3, 5).transpose(1, 2), None, torch.ones(3)), "channels"),
    (lambda: pr.block_norm(None, torch.zeros(2, 5, 3), None, torch.ones(3), z_dtype=torch.float16), "z_dtype"),
    (lambda: pr.block_norm(torch.zeros(2, 3, 5), torch.zeros(2, 5, 3), None, torch.ones(3)), "w_post"),
    (lambda: pr.block_norm(None, torch.zeros(2, 5, 3), None, torch.ones(3)), "GPU"),
    (lambda: pr.block_norm_adjoint(None, torch.zeros(2, 5, 3), None, torch.ones(3), torch.zeros(2, 5), None, None), "rstd"),
    (lambda: pr.block_norm_adjoint(None, torch.zeros(2, 5, 3), None, torch.ones(3), torch.zeros(2, 2, 5),
                                   torch.zeros(2, 5, 3).bfloat16(), None), "gy"),
    (lambda: pr.token_logprobs(torch.zeros(2, 9, dtype=torch.float64), torch.zeros(2, dtype=torch.int64)), "logits"),
    (lambda: pr.token_logprobs(torch.zeros(9, 2).t(), torch.zeros(2, dtype=torch.int64)), "contiguous"),
    (lambda: pr.token_logprobs(torch.zeros(2, 9), torch.zeros(2, dtype=torch.int32)), "int64"),
    (lambda: pr.token_logprobs(torch.zeros(2, 9), torch.zeros(2, dtype=torch.int64), top=65), "top"),
    (lambda: pr.token_logprobs(torch.zeros(2, 9), torch.zeros(2, dtype=torch.int64)), "GPU"),
    (lambda: pr.token_logprobs_adjoint(torch.zeros(2, 9), torch.zeros(2, dtype=torch.int64), None), "lse"),
    (lambda: pr.token_logprobs_adjoint(torch.zeros(2, 9), torch.zeros(2, dtype=torch.int64), torch.zeros(2),
                                       g_entropy=torch.zeros(2)), "entropy"),
    (lambda: pr.token_logprobs_adjoint(torch.zeros(2, 9), torch.zeros(2, dtype=torch.int64), torch.zeros(2),
                                       out=torch.zeros(2, 9).bfloat16()), "out"),
])
def test_binding(call, message):
    for _ in range(2):  # the second time as well: a refusal is not remembered as a plan
        with pytest.raises(ValueError, match=message):
            call()

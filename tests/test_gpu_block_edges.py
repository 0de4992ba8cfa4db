"""The block boundary at the edges of what its kernels reach: long rows without
states, offsets near 32 bits, more tiles than a dispatch can count, time-major
planes that give every compute unit work.

Tolerances as in test_gpu_block.py: 2^-24 (D / 64 + 64) of the largest value."""
import numpy as np
import pytest
import torch

from nonlinear_rnn_amd import pararnn as pr
from tests.gpu_util import DEV
from tests.test_gpu_block import F, H, check, inputs

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24


def normed(x, w, eps=1e-6):
    x = x.double()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.double()


def near(got, want, D):
    assert float((got.double() - want).abs().max()) <= EPS * (D / 64 + 64) * max(1.0, float(want.abs().max()))


def test_the_first_norm_of_a_long_row_is_the_short_ones():
    """Without states their strides say nothing: 2^29 elements a row run the kernel
    that rows of 4096 steps run, to the same bits."""
    T, D = 2 ** 18, 2048
    x = torch.empty((1, T, D), dtype=H, device=DEV).normal_()
    w = torch.rand(D, device=DEV) + 0.5
    _, z, rstd = pr.block_norm(None, x, None, w, z_dtype=H)
    gz = torch.empty((1, T, D), dtype=H, device=DEV).normal_()
    dx = pr.block_norm_adjoint(None, x, None, w, rstd, None, gz)["dx"]
    for t in (0, T // 2, T - 2 ** 14):
        part = x[:, t:t + 2 ** 14]
        _, zp, rp = pr.block_norm(None, part, None, w, z_dtype=H)
        assert torch.equal(z[:, t:t + 2 ** 14], zp) and torch.equal(rstd[1:, :, t:t + 2 ** 14], rp[1:])
        dp = pr.block_norm_adjoint(None, part, None, w, rp, None, gz[:, t:t + 2 ** 14])["dx"]
        assert torch.equal(dx[:, t:t + 2 ** 14], dp)
    near(pr.block_norm(None, x[:, -64:], None, w, z_dtype=F)[1], normed(x[:, -64:], w), D)


@pytest.mark.parametrize("D", [1, 2])
def test_more_tiles_than_a_dispatch_counts(D):
    """2^28 steps and a few of one or two channels."""
    T = 2 ** 28 + 5
    x = torch.empty((1, T, D), device=DEV).normal_()
    w = torch.rand(D, device=DEV) + 0.5
    _, z, rstd = pr.block_norm(None, x, None, w, z_dtype=F, eps=1e-2)
    ends = [slice(0, 4099), slice(T - 4099, T)]
    for s in ends:
        near(z[:, s], normed(x[:, s], w, 1e-2), D)
    got = pr.block_norm_adjoint(None, x, None, w, rstd, None, z)
    for s in ends:
        n2, q = x[:, s].double() * rstd[1, :, s, None], z[:, s].double() * w.double()
        want = rstd[1, :, s, None].double() * (q - n2 * (q * n2).mean(-1, keepdim=True))
        near(got["dx"][:, s], want, D)
    dw = sum(float((z[:, i:i + 2 ** 24].double() * x[:, i:i + 2 ** 24].double()
                    * rstd[1, :, i:i + 2 ** 24, None]).sum()) for i in range(0, T, 2 ** 24))
    # chains of at most T / (512 2 D) steps of positive terms, rounded at random; all of them at worst
    assert abs(float(got["dw_pre"].double().sum()) - dw) <= EPS * 2 ** 19 * abs(dw)


@pytest.mark.parametrize("dt", [F, H])
def test_offsets_near_32_bits(dt):
    """Channels and steps as far apart as the register kernels reach, and one
    element further: there the strip kernels run."""
    B, T, D = 1, 20, 2
    for far, step in ((2 ** 28 - 4, 2 ** 25 - 1), (2 ** 28 - 3, 2 ** 25)):
        c = inputs(B, T, D, dt, dt)
        big = torch.zeros(far + T + 64, device=DEV)
        c["h"] = torch.as_strided(big, (B, D, T), (2 * far, far, 1)).copy_(c["h"])
        gates = torch.zeros(far + T + 64, dtype=dt, device=DEV)
        c["gate"] = torch.as_strided(gates, (B, D, T), (2 * far, far, 1)).copy_(c["gate"])
        for name in ("x", "gy"):
            rows = torch.zeros(T * step + D, dtype=dt, device=DEV)
            c[name] = torch.as_strided(rows, (B, T, D), (T * step, step, 1)).copy_(c[name])
        check(c, F)


def test_wide_rows_near_32_bits():
    """4096 channels of as many steps as the offsets allow, and of more: the last
    steps of each against float64."""
    D = 4096
    for T in (131071, 131200):
        h, x = torch.empty((1, D, T), device=DEV).normal_(), torch.empty((1, T, D), device=DEV).normal_()
        gate = torch.empty((1, D, T), dtype=H, device=DEV).normal_()
        w = torch.rand(D, device=DEV) + 0.5
        y, z, rstd = pr.block_norm(h, x, w, w, gate=gate, scale=0.5, z_dtype=F)
        s = slice(T - 70, T)
        g = gate[..., s].double().transpose(1, 2)
        v = h[..., s].double().transpose(1, 2) * g * torch.sigmoid(g)
        want = x[:, s].double() + 0.5 * normed(v, w)
        near(y[:, s], want, D)
        near(z[:, s], normed(want, w), D)
        got = pr.block_norm_adjoint(h, x, w, w, rstd, x, z, gate=gate, scale=0.5)
        r1, r2 = (rstd[i, :, s, None].double() for i in (0, 1))
        n1, n2, q = v * r1, want * r2, z[:, s].double() * w.double()
        dx = x[:, s].double() + r2 * (q - n2 * (q * n2).mean(-1, keepdim=True))
        near(got["dx"][:, s], dx, D)
        p = 0.5 * dx * w.double()
        dv = r1 * (p - n1 * (p * n1).mean(-1, keepdim=True))
        near(got["dh"][..., s], (dv * g * torch.sigmoid(g)).transpose(1, 2), 8 * D)
        del h, x, gate, y, z, got


@pytest.mark.parametrize("B,T,D", [(3, 2741, 65), (2, 4103, 130), (2, 4101, 520), (1, 8195, 770), (2, 4103, 1030),
                                   (2, 2053, 2050), (2, 2053, 4096)])
@pytest.mark.parametrize("dt", [F, H])
def test_time_major_planes_with_work_for_every_unit(B, T, D, dt):
    check(inputs(B, T, D, dt, F if D % 4 else dt, layout="time"), F if D % 5 else H)


@pytest.mark.parametrize("B,T,D,layout", [(1, 1, 8192, "channel"), (2, 9, 6001, "channel"), (1, 700, 8191, "channel"),
                                          (2, 30, 5120, "time"), (1, 5, 8192, "padded"), (1, 33, 8193, "channel")])
@pytest.mark.parametrize("gdt,xdt,zdt", [(F, F, F), (H, F, H), (H, H, H)])
def test_more_than_4096_channels(B, T, D, layout, gdt, xdt, zdt):
    check(inputs(B, T, D, gdt, xdt, layout=layout), zdt)


def test_more_than_4096_channels_with_parts_left_out():
    for use in (("gy", "gz"), ("h", "gy"), ("h", "gate", "gz")):
        check(inputs(1, 21, 7000), use=use)


def test_more_than_4096_channels_repeat():
    """Tiles of 8192 channels have one workgroup's order of sums: the same bits each
    time, and for a row among others as by itself."""
    c = inputs(2, 40, 8000, H, F)
    run = [pr.block_norm(c["h"], c["x"], c["wp"], c["wn"], gate=c["gate"]) for _ in range(2)]
    alone = pr.block_norm(c["h"][1:], c["x"][1:], c["wp"], c["wn"], gate=c["gate"][1:])
    for a, b in zip(*run):
        assert torch.equal(a, b)
    y, z, rstd = run[0]
    for a, b in zip((y[1:], z[1:], rstd[:, 1:]), alone):
        assert torch.equal(a, b)

"""The block boundary on the GPU against the float64 oracle.

Tolerance.  A mean of D terms is a chain of at most D / 64 additions in a lane
and a tree across lanes: within 2^-24 (D / 64 + 16) of its magnitude; the
elementwise part adds under 48 roundings.  Outputs are sums of terms no larger
than the reference's largest value times the norms' gains (below 8 here), so
tol = 2^-24 (D / 64 + 64) max(1, |reference|), and half an ulp for bf16.  Sums
over steps: their terms' magnitudes by 2^-24 (64 + D / 64 + steps / 64)."""
import numpy as np
import pytest
import torch

from nonlinear_rnn_amd import autograd as pag
from nonlinear_rnn_amd import pararnn as pr
from oracle import language as ref
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24
F, H = torch.float32, torch.bfloat16


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def dev(x, dt=F):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV).to(dt)


def close(got, exact, D, bf16=False, scale=None):
    exact = np.asarray(exact)
    tol = EPS * (D / 64 + 64) * max(1.0, np.abs(exact).max(initial=0.0) if scale is None else scale)
    diff = np.abs(f64(got) - exact)
    assert got.shape == exact.shape
    assert (diff <= tol + (2.0 ** -8 * np.abs(exact) if bf16 else 0)).all(), (float(diff.max()), tol)


def inputs(B, T, D, gdt=F, xdt=F, seed=0, layout="channel"):
    r = np.random.default_rng(seed + 7 * T + D)

    def plane(dt):
        x = dev(r.standard_normal((B, D, T)), dt)
        if layout == "time":
            return x.transpose(1, 2).contiguous().transpose(1, 2)
        if layout == "padded":
            return torch.empty((B, D + 1, T + 3), dtype=dt, device=DEV)[:, 1:, 1:T + 1].copy_(x)
        return x
    x = dev(2 * r.standard_normal((B, T, D)), xdt)
    if layout == "padded":
        x = torch.empty((B, T + 1, D + 5), dtype=xdt, device=DEV)[:, :T, 3:D + 3].copy_(x)
    gy = torch.empty_strided(x.shape, x.stride(), dtype=xdt, device=DEV).copy_(dev(r.standard_normal((B, T, D))))
    return dict(h=plane(F), gate=plane(gdt), x=x, wp=dev(1 + 0.2 * r.standard_normal(D)),
                wn=dev(1 + 0.2 * r.standard_normal(D)), gy=gy, gz=r.standard_normal((B, T, D)))


def check(c, zdt=F, scale=0.5, eps=1e-5, use=("h", "gate", "gy", "gz")):
    B, T, D = c["x"].shape
    h, gate = (c[k] if k in use else None for k in ("h", "gate"))
    kw = dict(gate=gate, scale=scale)
    y, z, rstd = pr.block_norm(h, c["x"], c["wp"], c["wn"], eps=eps, z_dtype=zdt, **kw)
    nx = [f64(h), f64(c["x"]), f64(c["wp"]), f64(c["wn"])]
    ey, ez, er = ref.block_norm(*nx, f64(gate), scale, eps)
    xh, gh = c["x"].dtype == H, gate is not None and gate.dtype == H
    close(y, ey, D, xh)
    close(z, ez, D, zdt == H)
    assert y.dtype == c["x"].dtype and z.dtype == zdt
    for i in (0, 1) if h is not None else (1,):
        assert (np.abs(f64(rstd[i]) - er[i]) <= EPS * (D / 64 + 24) * er[i]).all()
    gy = c["gy"] if "gy" in use else None
    gz = dev(c["gz"], zdt) if "gz" in use else None
    got = pr.block_norm_adjoint(h, c["x"], c["wp"], c["wn"], rstd, gy, gz, **kw)
    want = ref.block_norm_adjoint(*nx, f64(gy), f64(gz), f64(gate), scale, eps)
    close(got["dx"], want["dx"], D, xh)
    # the norms divide by the root mean square of their input, which may be small
    gain = max(1.0, er.max())
    if h is not None:
        close(got["dh"], want["dh"], D, False, gain * max(1.0, np.abs(want["dx"]).max()) * 8)
        assert got["dh"].stride() == h.stride()
    if gate is not None:
        close(got["dgate"], want["dgate"], D, gh, gain * max(1.0, np.abs(want["dx"]).max()) * 8)
    for name in ("dw_post", "dw_pre"):
        if want[name] is None:
            assert got[name] is None
            continue
        tol = EPS * (64 + D / 64 + B * T / 64) * np.maximum(1.0, want["dw_terms"])
        assert (np.abs(f64(got[name]) - want[name]) <= tol).all(), name


SHAPES = [(1, 1, 1), (3, 1, 64), (2, 1, 1000), (1, 2, 130), (2, 5, 7), (1, 16, 256), (2, 17, 96),
          (1, 31, 2000), (3, 64, 65), (1, 50, 1024), (2, 33, 4096), (1, 9, 4100), (1, 20, 9001)]


@pytest.mark.parametrize("gdt,xdt,zdt", [(F, F, F), (H, F, H), (H, H, H), (F, H, F)])
@pytest.mark.parametrize("B,T,D", SHAPES)
def test_block(B, T, D, gdt, xdt, zdt):
    check(inputs(B, T, D, gdt, xdt), zdt)


# enough steps for the longest tiles, at every width of theirs
@pytest.mark.parametrize("B,T,D", [(3, 2741, 7), (3, 2741, 65), (2, 4103, 130), (2, 4103, 192), (1, 8209, 301),
                                   (2, 4101, 520), (1, 8195, 770), (2, 4103, 1030), (1, 8200, 1540),
                                   (2, 2053, 2050), (2, 2053, 3333)])
def test_long_tiles(B, T, D):
    check(inputs(B, T, D, H if D % 2 else F, H if D % 3 else F), H if D % 5 else F)


@pytest.mark.parametrize("layout", ["time", "padded"])
@pytest.mark.parametrize("B,T,D", [(2, 1, 100), (2, 5, 70), (2, 40, 513), (1, 21, 4096)])
@pytest.mark.parametrize("dt", [F, H])
def test_layouts(B, T, D, layout, dt):
    check(inputs(B, T, D, dt, dt, layout=layout), H)


@pytest.mark.parametrize("use", [("h", "gy", "gz"), ("gy", "gz"), ("gz",), ("gy",), ("h", "gate", "gy"),
                                 ("h", "gate", "gz"), ("h", "gate")])
@pytest.mark.parametrize("B,T,D", [(2, 1, 70), (2, 18, 300), (1, 16, 2048)])
def test_parts_left_out(B, T, D, use):
    check(inputs(B, T, D), use=use)


def test_many_steps():
    """More tiles than workgroups, so that each keeps its weight gradients over several."""
    check(inputs(5, 7001, 72, H, F), H)


def test_zero_rows_and_gates():
    c = inputs(2, 20, 300)
    c["h"][:, :, 3] = 0          # nothing to norm: eps alone divides
    c["gate"][:, :, 5] = -1e4    # a gate that lets nothing through
    c["gate"][:, :, 6] = 1e4
    c["x"][1, 7] = 0
    check(c)
    y, _, _ = pr.block_norm(c["h"], c["x"], c["wp"], c["wn"], gate=c["gate"])
    assert torch.equal(y[:, 3], c["x"][:, 3]) and torch.equal(y[:, 5], c["x"][:, 5])


def test_nan_stays_in_its_step():
    c = inputs(2, 20, 300)
    c["h"][1, 17, 4] = float("nan")
    y, z, _ = pr.block_norm(c["h"], c["x"], c["wp"], c["wn"], gate=c["gate"], z_dtype=F)
    assert torch.isnan(y[1, 4]).all() and torch.isnan(z[1, 4]).all()
    assert int(torch.isnan(z).sum()) == 300


def test_empty_sizes():
    w = torch.ones(8, device=DEV)
    for shape in ((0, 5, 8), (3, 0, 8)):
        x, h = torch.empty(shape, device=DEV), torch.empty((shape[0], 8, shape[1]), device=DEV)
        y, z, rstd = pr.block_norm(h, x, w, w)
        assert y.shape == z.shape == shape
        got = pr.block_norm_adjoint(h, x, w, w, rstd, x, z)
        assert not got["dw_post"].any() and not got["dw_pre"].any()


def test_offsets_past_32_bits():
    far = 2 ** 30 + 8
    B, T, D = 1, 20, 3
    c = inputs(B, T, D)
    big = torch.zeros(2 * far + 64, device=DEV)
    strides = (3 * far, far, 1)
    h = torch.as_strided(big, (B, D, T), strides).copy_(c["h"])
    gate = torch.as_strided(big, (B, D, T), strides, 32).copy_(c["gate"])
    a = pr.block_norm(h, c["x"], c["wp"], c["wn"], gate=gate, z_dtype=F)
    b = pr.block_norm(c["h"], c["x"], c["wp"], c["wn"], gate=c["gate"], z_dtype=F)
    for p, q in zip(a, b):
        close(p, f64(q), D)
    c["h"], c["gate"] = h, gate
    check(c)


def test_another_stream_and_repeatable():
    c = inputs(3, 400, 520, H, F)
    gz = dev(c["gz"], H)
    s = torch.cuda.Stream()

    def run(**kw):
        y, z, rstd = pr.block_norm(c["h"], c["x"], c["wp"], c["wn"], gate=c["gate"], **kw)
        b = pr.block_norm_adjoint(c["h"], c["x"], c["wp"], c["wn"], rstd, c["gy"], gz, gate=c["gate"], **kw)
        return [y, z, rstd] + [b[k] for k in sorted(b)]
    one = run()
    torch.cuda.synchronize()
    two = run(stream=s)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(one, two))


@pytest.mark.parametrize("with_h", [True, False])
def test_autograd(with_h):
    c = inputs(2, 21, 70)
    leaves = {k: c[k].clone().requires_grad_(True) for k in ("h", "gate", "x", "wp", "wn")}
    h, gate = (leaves["h"], leaves["gate"]) if with_h else (None, None)
    y, z = pag.block_norm(h, leaves["x"], leaves["wp"] if with_h else None, leaves["wn"], gate=gate,
                          scale=0.5, z_dtype=F)
    gz = dev(c["gz"])
    (y.sum() + (z * gz).sum()).backward()
    want = ref.block_norm_adjoint(f64(h), f64(c["x"]), f64(c["wp"]), f64(c["wn"]), np.ones(y.shape),
                                  f64(gz), f64(gate), 0.5)
    names = dict(x="dx", wn="dw_pre", **(dict(h="dh", gate="dgate", wp="dw_post") if with_h else {}))
    for leaf, name in names.items():
        close(leaves[leaf].grad, want[name], 70, scale=8 * max(1.0, np.abs(want[name]).max()))

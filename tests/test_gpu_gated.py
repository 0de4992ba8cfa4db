"""The gated linear recurrence on the GPU against the float64 oracle.

Tolerance.  A step rounds the decay a (1 - m: half an ulp), the product with
the state, and the input term (under 8 ulp: two gates, a root, two products).
An error of one step fades by a per step, so with the largest decay A of the
inputs the state is within 2^-24 (2 |h| + 8 |b|) / (1 - A) of the exact one, and
each level of the scan (under 32 of them) adds at most an ulp of the state:
tol = 2^-24 (16 / (1 - A) + 32) max(1, |h|, |b|).  The backward recurrence has
the same decays; its gradients are products of G, the states and the inputs,
with at most 64 more roundings.  bf16 gradients add half an ulp, 2^-9."""
import numpy as np
import pytest
import torch

from nonlinear_rnn_amd import autograd as pag
from nonlinear_rnn_amd import pararnn as pr
from oracle import language as ref
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def case(B, T, D, dtype=torch.float32, layout="channel", docs=None, h0=True, seed=0, power=8.0):
    r = np.random.default_rng(seed + 1000 * T + D)

    def plane(std=1.0, dt=torch.float32):
        x = torch.from_numpy(std * r.standard_normal((B, D, T))).to(DEV).to(dt)
        if layout == "time":
            return x.transpose(1, 2).contiguous().transpose(1, 2)
        if layout == "padded":  # rows of channels at odd offsets
            y = torch.empty((B, D + 1, T + 3), dtype=dt, device=DEV)[:, :D, 1:T + 1]
            return y.copy_(x)
        if layout == "mixed":  # batch innermost
            return x.permute(1, 2, 0).contiguous().permute(2, 0, 1)
        return x
    decay = 0.9 + 0.099 * r.random(D)
    lam = torch.from_numpy(np.log(np.expm1(-np.log(decay) / power))).float().to(DEV)
    resets = None
    if docs == "all":
        resets = torch.ones((B, T), dtype=torch.bool, device=DEV)
    elif docs is not None:
        resets = torch.from_numpy(r.random((B, T)) < docs).to(DEV)
    h0 = torch.from_numpy(r.standard_normal((B, D))).float().to(DEV) if h0 else None
    return dict(u=[plane(dt=dtype) for _ in range(3)], lam=lam, h0=h0, resets=resets,
                gh=plane(), gl=torch.from_numpy(r.standard_normal((B, D))).float().to(DEV), power=power)


def tolerance(c):
    l, _ = ref._log_decay(f64(c["u"][0]), f64(c["lam"]), c["power"])
    return EPS * (16 / (-np.expm1(l.max(initial=-1.0))) + 32)


def close(got, exact, tol, bf16=False):
    got = f64(got)
    assert got.shape == exact.shape
    assert (np.abs(got - exact) <= tol + (2.0 ** -8 * np.abs(exact) if bf16 else 0)).all(), (
        float(np.abs(got - exact).max(initial=0.0)), tol)


SHAPES = [(1, 1, 1), (2, 1, 130), (1, 2, 3), (3, 7, 65), (2, 63, 5), (2, 64, 64), (1, 65, 2),
          (3, 4, 20), (2, 16, 70), (2, 17, 33), (2, 32, 9), (1, 33, 130), (2, 128, 21),
          (2, 300, 33), (1, 513, 9), (2, 1025, 3), (1, 4100, 2), (1, 20011, 1), (5, 129, 200)]


@pytest.mark.parametrize("layout", ["channel", "time", "padded", "mixed"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,T,D", SHAPES)
def test_scan_and_adjoint(B, T, D, dtype, layout):
    c = case(B, T, D, dtype, layout, docs=0.02 if D % 2 else None, h0=D != 5)
    h, last = pr.gated_scan(c["u"], c["lam"], c["h0"], power=c["power"], resets=c["resets"])
    u = [f64(p) for p in c["u"]]
    exact = ref.gated_scan(u, f64(c["lam"]), f64(c["h0"]), c["power"], f64(c["resets"]))
    scale = max(1.0, np.abs(exact).max(), max(np.abs(p).max() for p in u))
    close(h, exact, tolerance(c) * scale)
    assert torch.equal(last, h[..., -1].contiguous())
    gh = torch.empty_strided(h.shape, h.stride(), device=DEV).copy_(c["gh"])
    got = pr.gated_scan_adjoint(c["u"], c["lam"], c["h0"], h, gh, gh_last=c["gl"], power=c["power"],
                                resets=c["resets"])
    want = ref.gated_scan_adjoint(u, f64(c["lam"]), f64(c["h0"]), f64(h), f64(gh), c["power"],
                                  f64(c["resets"]), f64(c["gl"]))
    tol = (tolerance(c) + 64 * EPS) * max(1.0, want["G_max"])
    for g in range(3):
        assert got["du"][g].dtype == dtype and got["du"][g].stride() == c["u"][g].stride()
        close(got["du"][g], want["du"][g], tol * scale, dtype == torch.bfloat16)
    close(got["dh0"], want["dh0"], tol)
    assert (np.abs(f64(got["dlam"]) - want["dlam"]) <= tol * np.maximum(1.0, want["dlam_terms"])).all()


# many parts of one channel, of few and of some, a part with one step, and
# channels that fill the device
PARTS = [(1, 290000, 1, "channel"), (3, 12289, 5, "channel"), (1, 4097, 300, "padded"),
         (1, 30000, 70, "time"), (3, 65, 130, "mixed"), (2, 64, 100, "time"), (1, 40, 131100, "time"),
         (1, 4099, 2049, "channel"), (1, 6139, 2048, "padded"),
         (1, 600, 2100, "channel")]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,T,D,layout", PARTS)
def test_parts_of_the_time_axis(B, T, D, layout, dtype):
    test_scan_and_adjoint(B, T, D, dtype, layout)


@pytest.mark.parametrize("B,T,D,layout", PARTS[:5])
def test_same_bits_every_time(B, T, D, layout):
    c = case(B, T, D, torch.bfloat16, layout, docs=0.0002)
    first = None
    for _ in range(4):
        h, last = pr.gated_scan(c["u"], c["lam"], c["h0"], power=c["power"], resets=c["resets"])
        g = pr.gated_scan_adjoint(c["u"], c["lam"], c["h0"], h, None, gh_last=c["gl"], power=c["power"],
                                  resets=c["resets"])
        now = [h, last, *g["du"], g["dh0"], g["dlam"]]
        first = first or now
        assert all(torch.equal(x, y) for x, y in zip(now, first))


@pytest.mark.parametrize("layout", ["channel", "time"])
def test_every_step_a_new_document(layout):
    c = case(2, 150, 66, layout=layout, docs="all")
    h, _ = pr.gated_scan(c["u"], c["lam"], c["h0"], power=c["power"], resets=c["resets"])
    other, _ = pr.gated_scan(c["u"], c["lam"], None, power=c["power"], resets=c["resets"])
    assert torch.equal(h, other)  # nothing of h0 is left
    exact = ref.gated_scan([f64(p) for p in c["u"]], f64(c["lam"]), f64(c["h0"]), c["power"], f64(c["resets"]))
    close(h, exact, 16 * EPS * max(1.0, np.abs(exact).max()))
    got = pr.gated_scan_adjoint(c["u"], c["lam"], c["h0"], h, None, gh_last=c["gl"], power=c["power"],
                                resets=c["resets"])
    assert not got["dh0"].any() and not got["du"][0][..., :-1].any()


def test_cut_sequence_is_the_whole_one():
    """Two halves, the second from the first's last state, and their gradients."""
    c = case(2, 700, 40)
    h, last = pr.gated_scan(c["u"], c["lam"], c["h0"], power=c["power"])
    halves = [[p[..., s].contiguous() for p in c["u"]] for s in (slice(0, 333), slice(333, 700))]
    h1, l1 = pr.gated_scan(halves[0], c["lam"], c["h0"], power=c["power"])
    h2, l2 = pr.gated_scan(halves[1], c["lam"], l1, power=c["power"])
    tol = 2 * tolerance(c) * max(1.0, float(h.abs().max()))
    close(torch.cat([h1, h2], -1), f64(h), tol)
    close(l2, f64(last), tol)
    whole = pr.gated_scan_adjoint(c["u"], c["lam"], c["h0"], h, c["gh"], power=c["power"])
    b2 = pr.gated_scan_adjoint(halves[1], c["lam"], l1, h2, c["gh"][..., 333:].contiguous(), power=c["power"])
    b1 = pr.gated_scan_adjoint(halves[0], c["lam"], c["h0"], h1, c["gh"][..., :333].contiguous(),
                               gh_last=b2["dh0"], power=c["power"])
    tol *= 50  # gradients summed over the memory of the recurrence
    close(b1["dh0"], f64(whole["dh0"]), tol)
    close(torch.cat([b1["du"][0], b2["du"][0]], -1), f64(whole["du"][0]), tol)


@pytest.mark.parametrize("T", [1, 70, 3000])
def test_extreme_gates_stay_finite(T):
    """Gates that saturate both ways: the decay underflows to 1 and to 0, the
    gain to 0, and no gradient divides by it."""
    B, D = 1, 70
    r = np.random.default_rng(T)
    extremes = np.array([-1e4, -200.0, -90.0, -40.0, 0.0, 40.0, 200.0, 1e4], np.float32)
    u = [torch.from_numpy(r.choice(extremes, (B, D, T))).to(DEV) for _ in range(2)]
    u.append(torch.from_numpy(r.standard_normal((B, D, T))).float().to(DEV))
    lam = torch.linspace(-120.0, 120.0, D, device=DEV)
    h, _ = pr.gated_scan(u, lam, None)
    gh = torch.ones_like(h)
    got = pr.gated_scan_adjoint(u, lam, None, h, gh)
    exact = ref.gated_scan([f64(p) for p in u], f64(lam), None, 8.0)
    close(h, exact, EPS * 16 * max(1.0, np.abs(exact).max()) * T)
    for t in got["du"] + [got["dlam"], got["dh0"]]:
        assert torch.isfinite(t).all()
    want = ref.gated_scan_adjoint([f64(p) for p in u], f64(lam), None, f64(h), f64(gh), 8.0)
    for g in range(3):
        close(got["du"][g], want["du"][g], 64 * EPS * T * max(1.0, np.abs(exact).max()) * max(1.0, want["G_max"]))


def test_nan_reaches_its_own_channel_only():
    c = case(2, 200, 5)
    c["u"][2][1, 3, 50] = float("nan")
    h, _ = pr.gated_scan(c["u"], c["lam"], c["h0"], power=c["power"])
    bad = torch.isnan(h)
    assert bad[1, 3, 50:].all() and int(bad.sum()) == 150


def test_empty_sizes():
    lam = torch.zeros(4, device=DEV)
    h0, gl = torch.randn(3, 4, device=DEV), torch.randn(3, 4, device=DEV)
    u = [torch.empty((3, 4, 0), device=DEV)] * 3
    h, last = pr.gated_scan(u, lam, h0)
    assert h.shape == (3, 4, 0) and torch.equal(last, h0)
    got = pr.gated_scan_adjoint(u, lam, h0, h, None, gh_last=gl)
    assert torch.equal(got["dh0"], gl) and not got["dlam"].any()
    u = [torch.empty((0, 4, 6), device=DEV)] * 3
    h, last = pr.gated_scan(u, lam)
    got = pr.gated_scan_adjoint(u, lam, None, h, None)
    assert last.shape == (0, 4) and not got["dlam"].any()


@pytest.mark.parametrize("layout", ["channel", "time"])
def test_offsets_past_32_bits(layout):
    """Channels (or steps) 2^30 + 8 elements apart: the last plane's elements lie
    past 2^31 elements and 2^32 bytes."""
    far = 2 ** 30 + 8
    B, D, T = 1, (3 if layout == "channel" else 70), (70 if layout == "channel" else 3)
    big = torch.zeros(2 * far + 256, dtype=torch.float32, device=DEV)
    stride = (3 * far, far, 1) if layout == "channel" else (3 * far, 1, far)
    c = case(B, T, D)
    u = [torch.as_strided(big, (B, D, T), stride, 70 * g).copy_(p) for g, p in enumerate(c["u"])]
    out = torch.as_strided(torch.zeros_like(big), (B, D, T), stride)
    h, _ = pr.gated_scan(u, c["lam"], c["h0"], power=c["power"], out=out)
    want, _ = pr.gated_scan(c["u"], c["lam"], c["h0"], power=c["power"])
    tol = 2 * tolerance(c) * max(1.0, float(want.abs().max()))
    close(h, f64(want), tol)
    gh = torch.as_strided(torch.zeros_like(big), (B, D, T), stride).copy_(c["gh"])
    got = pr.gated_scan_adjoint(u, c["lam"], c["h0"], h, gh, power=c["power"])
    exact = ref.gated_scan_adjoint([f64(p) for p in c["u"]], f64(c["lam"]), f64(c["h0"]), f64(h),
                                   f64(c["gh"]), c["power"])
    tol = (tolerance(c) + 64 * EPS) * max(1.0, exact["G_max"]) * max(1.0, np.abs(f64(h)).max(), 4.0)
    for g in range(3):
        close(got["du"][g], exact["du"][g], tol)


def test_another_stream_and_repeatable():
    c = case(2, 5000, 9)
    s = torch.cuda.Stream()
    first = pr.gated_scan(c["u"], c["lam"], c["h0"], power=c["power"])[0]
    back = pr.gated_scan_adjoint(c["u"], c["lam"], c["h0"], first, c["gh"], power=c["power"])
    torch.cuda.synchronize()
    h, _ = pr.gated_scan(c["u"], c["lam"], c["h0"], power=c["power"], stream=s)
    again = pr.gated_scan_adjoint(c["u"], c["lam"], c["h0"], h, c["gh"], power=c["power"], stream=s)
    s.synchronize()
    assert torch.equal(first, h)
    for a, b in zip(back["du"] + [back["dlam"], back["dh0"]], again["du"] + [again["dlam"], again["dh0"]]):
        assert torch.equal(a, b)


def test_autograd():
    c = case(2, 90, 6, docs=0.05)
    u = [p.clone().requires_grad_(True) for p in c["u"]]
    lam, h0 = c["lam"].clone().requires_grad_(True), c["h0"].clone().requires_grad_(True)
    h, last = pag.gated_scan(u, lam, h0, power=c["power"], resets=c["resets"])
    (h.sum() + (last * c["gl"]).sum()).backward()  # the sum's gradient is one broadcast element
    want = ref.gated_scan_adjoint([f64(p) for p in u], f64(lam), f64(h0), f64(h), np.ones(h.shape),
                                  c["power"], f64(c["resets"]), f64(c["gl"]))
    tol = (tolerance(c) + 64 * EPS) * max(1.0, want["G_max"]) * max(1.0, float(h.abs().max()), 4.0)
    for g in range(3):
        close(u[g].grad, want["du"][g], tol)
    close(h0.grad, want["dh0"], tol)
    assert (np.abs(f64(lam.grad) - want["dlam"]) <= tol * np.maximum(1.0, want["dlam_terms"])).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,D", [(1, 1), (3, 64), (2, 1000), (70, 257)])
def test_step(B, D, dtype):
    r = np.random.default_rng(B * D)
    pool = B + 3
    u = torch.from_numpy(r.standard_normal((B, 3 * D))).to(DEV).to(dtype)
    u = [u[:, g * D:(g + 1) * D] for g in range(3)]
    lam = torch.from_numpy(r.standard_normal(D)).float().to(DEV)
    states = torch.from_numpy(r.standard_normal((pool, D))).float().to(DEV)
    slots = torch.from_numpy(r.permutation(pool)[:B].astype(np.int32)).to(DEV)
    if B > 2:
        slots[1], slots[2] = -1, pool  # idle: no slot, and one past the pool
    old = states.clone()
    new = pr.gated_step(u, lam, states, slots=slots)
    want = old.clone().double().cpu().numpy()
    for b, s in enumerate(slots.tolist()):
        if not 0 <= s < pool:
            assert not new[b].any()
            continue
        exact = ref.gated_scan([f64(p)[b][None, :, None] for p in u], f64(lam), f64(old[s])[None], 8.0)[0, :, 0]
        close(new[b], exact, 32 * EPS * 4)
        want[s] = f64(new[b])
    assert np.array_equal(f64(states), want)


def test_step_follows_the_scan():
    """A prompt through the scan, then token by token: the same states."""
    c = case(3, 40, 50)
    h, _ = pr.gated_scan(c["u"], c["lam"], c["h0"], power=c["power"])
    states = h[..., 29].contiguous()
    for t in range(30, 40):
        out = pr.gated_step([p[..., t].contiguous() for p in c["u"]], c["lam"], states, power=c["power"])
        close(out, f64(h[..., t]), 2 * tolerance(c) * max(1.0, float(h.abs().max())))

"""The gated recurrence where its gates are at their ends, on the GPU: closed gates, gates that are NaN, decays next to
0 and infinite ones, against the 64-bit forms."""
from __future__ import annotations

import pytest
import torch

import tests.seq_ref as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def cf():
    import implicit_gemm_convolution_conv2d_b200 as mod
    return mod


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def ok(got, ref, bound, dtype, name):
    w = R.worst(got, ref, bound, dtype)
    assert w <= 1.0, f"{name}: {w:.3g} times what rounding allows"


def reference(x, r, i, decay, h0, cu, dy, dh_last):
    """(y, last, gradients by name, bounds) in 64 bits; the gradients by autograd."""
    leaves = {k: t.double().requires_grad_() for k, t in dict(x=x, r=r, i=i, decay=decay, h0=h0).items()}
    y, last = R.gated_scan(*leaves.values(), cu)
    loss = (y * dy.double()).sum() + (last * dh_last.double()).sum()
    grads = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))
    bound = R.scan_bounds(*(t.detach() for t in leaves.values()), cu, dy.double(), dh_last.double())
    return y.detach(), last.detach(), grads, bound


def both_passes(cf, x, r, i, decay, h0, cu, dy, dh_last):
    """(y, last, gradients by name) of the kernels, the backward pass from the forward pass's own states."""
    cuda = lambda t: None if t is None else cf.Act8(t.q.cuda(), t.scale.cuda(), t.dtype) if isinstance(t, cf.Act8) else t.cuda()  # noqa: E731
    whole = [cf.act8_unpack(cuda(t)) if isinstance(t, cf.Act8) else t.cuda() for t in (x, r, i)]
    x, r, i, decay, h0, cu, dy, dh_last = (cuda(t) for t in (x, r, i, decay, h0, cu, dy, dh_last))
    y, last, states = cf.gated_scan(*whole, decay, h0=h0, cu_seqlens=cu, save_states=True)
    grads = cf.gated_scan_grad(x, r, i, decay, dy, states, h0=h0, dh_last=dh_last, cu_seqlens=cu)
    return y, last, dict(zip(("x", "r", "i", "decay", "h0"), grads))


# ---- closed gates -------------------------------------------------------


@pytest.mark.parametrize("which", ["r", "i"])
@pytest.mark.parametrize("dtype", DT)
def test_closed_gates_keep_their_digits(cf, dtype, which):
    """Gates down to sigmoid(-80) = 1.8e-35: relative bounds, like those of open gates.  A channel's level is one of
    -20 .. -80 and decay at least 1, so that 1 - a^2 and each gradient are normal numbers of fp32."""
    g, dt, L, C = gen(60), DT[dtype], 150, 61
    x, r, i, dy = (normal(g, 2, L, C, dtype=dt) for _ in range(4))
    level = -20 - torch.arange(C).float()
    if which == "r":
        r = (r.float() * 0.1 + level).to(dt)
    else:
        i = (i.float() * 0.1 + level).to(dt)
    decay = 1 + torch.rand(C, generator=g)
    # without a state to begin from, what a closed input gate lets in is all there is
    h0, dh_last = torch.zeros(2, C), normal(g, 2, C)
    y, last, grads, bound = reference(x, r, i, decay, h0, None, dy, dh_last)
    gy, gl, gg = both_passes(cf, x, r, i, decay, h0, None, dy, dh_last)
    ok(gy, y, bound["y"], dt, "y")
    ok(gl, last, bound["last"], torch.float32, "h_last")
    for k, t in gg.items():
        ok(t, grads[k], bound["d" + k], torch.float32 if k in ("decay", "h0") else dt, "d" + k)
    # a token by itself
    pool = h0.cuda()
    z = cf.gated_scan_step(x[:, 0].cuda(), r[:, 0].cuda(), i[:, 0].cuda(), decay.cuda(), pool)
    ok(z, y[:, 0], bound["y"][:, 0], dt, "step")


@pytest.mark.parametrize("dtype", DT)
def test_gates_below_the_least_number_are_closed(cf, dtype):
    """Behind the least normal number of fp32 a gate is 0: nothing comes in, and the state stays as it is."""
    dt = DT[dtype]
    x, o = torch.full((1, 70, 6), 3.0, dtype=dt), torch.zeros(1, 70, 6, dtype=dt)
    shut = torch.tensor([-90.0, -200.0, -1000.0, -60000.0, float("-inf"), -89.0]).to(dt).expand(1, 70, 6)
    decay, h0 = torch.full((6,), 0.5), torch.full((1, 6), 2.0)
    y, last, grads = both_passes(cf, x, shut, o, decay, h0, None, torch.ones_like(x), torch.zeros(1, 6))
    assert (y == 2).all() and (last == 2).all() and (grads["x"] == 0).all() and (grads["r"] == 0).all() and (grads["h0"] == 70).all()
    y, last, grads = both_passes(cf, x, o, shut, decay, torch.zeros(1, 6), None, torch.ones_like(x), torch.zeros(1, 6))
    assert (y == 0).all() and (last == 0).all() and (grads["x"] == 0).all() and (grads["i"] == 0).all()


# ---- gates that are NaN -------------------------------------------------


@pytest.mark.parametrize("saved8", [False, True], ids=["", "8bit"])
@pytest.mark.parametrize("cu", [None, [0, 90, 90, 160, 290, 300]], ids=["batch", "packed"])
@pytest.mark.parametrize("which", ["r", "i", "both"])
@pytest.mark.parametrize("dtype", DT)
def test_gradients_beside_a_nan_gate(cf, dtype, which, cu, saved8):
    """A gate that is NaN makes NaN what the definition makes NaN, and nothing else: an input gate leaves the decays,
    and with them the gradients of earlier tokens, as they are."""
    g, dt, L, C = gen(61), DT[dtype], 300, 70
    shape = (L, C) if cu else (2, L, C)
    n = len(cu) - 1 if cu else 2
    x, r, i, dy = (normal(g, *shape, dtype=dt) for _ in range(4))
    for k, t in (("r", r), ("i", i)):
        if which in (k, "both"):
            flat = t.view(-1, L, C)
            flat[:, 100, 3::8] = float("nan")
            flat[-1, 201 if k == "i" else 215, 5::16] = float("nan")
            flat[0, 0, 1] = float("nan")
            flat[0, L - 1, 2] = float("nan")
    decay, h0, dh_last = torch.exp(torch.rand(C, generator=g) * 5 - 4), normal(g, n, C), normal(g, n, C)
    args = dict(x=x, r=r, i=i)
    if saved8:
        saved = {k: R.act8(t) for k, t in args.items()}
        whole = {k: R.act8_values(q, s).to(dt) for k, (q, s) in saved.items()}
        args = {k: cf.Act8(q, s, dt) for k, (q, s) in saved.items()}
        x, r, i = whole["x"], whole["r"], whole["i"]
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32)
    y, last, grads, bound = reference(x, r, i, decay, h0, c, dy, dh_last)
    gy, gl, gg = both_passes(cf, args["x"], args["r"], args["i"], decay, h0, c, dy, dh_last)
    assert not torch.isfinite(y).all()
    ok(gy, y, bound["y"], dt, "y")
    ok(gl, last, bound["last"], torch.float32, "h_last")
    for k, t in gg.items():
        # the states that the backward pass starts from are the kernel's own: off by no more than y's bound, as in the bounds
        ok(t, grads[k], bound["d" + k], torch.float32 if k in ("decay", "h0") else dt, "d" + k)


# ---- decays at their ends -----------------------------------------------


@pytest.mark.parametrize("dtype", DT)
def test_least_decays(cf, dtype):
    """Where 1 - a^2 is no normal number of fp32 it counts as 0, in both passes; beside that, the definition."""
    g, dt, L = gen(62), DT[dtype], 140
    decay = torch.tensor([0.0, 1e-45, 1e-42, 1e-39, 6e-39, 1.2e-38, 2e-38, 1e-37, 1e-30, 1e-20, 1e-9, 1e-3])
    C = len(decay)
    x, r, i, dy = (normal(g, 2, L, C, dtype=dt) for _ in range(4))
    r[0, 5::9, 8:10] = -40.0  # 1 - a^2 = 8e-48 and 8e-38
    h0, dh_last = normal(g, 2, C), normal(g, 2, C)
    y, last, grads, bound = reference(x, r, i, decay.clamp(min=1e-45), h0, None, dy, dh_last)
    gy, gl, gg = both_passes(cf, x, r, i, decay, h0, None, dy, dh_last)
    # what 1 - a^2 below the least number would have given: m < 2^-63, of each token
    rest = L * 2.0 ** -63 * x.double().abs().max()
    ok(gy, y, bound["y"] + rest, dt, "y")
    ok(gl, last, bound["last"] + rest, torch.float32, "h_last")
    for t in gg.values():
        assert torch.isfinite(t).all()
    most = (dy.double().abs().max() * L + dh_last.double().abs().max())  # of |G|
    ok(gg["x"], grads["x"], bound["dx"] + most * 2.0 ** -63, dt, "dx")
    ok(gg["i"], grads["i"], bound["di"] + most * rest, dt, "di")
    # decay s |G| a g |x| / m <= m |G x|, as 1 - a^2 <= 2 decay s
    ok(gg["r"], grads["r"], bound["dr"] + 2 * most * rest, dt, "dr")
    ok(gg["h0"], grads["h0"], bound["dh0"], torch.float32, "dh0")
    ok(gg["decay"][10:], grads["decay"][10:], bound["ddecay"][10:], torch.float32, "ddecay")
    assert (gg["x"][..., :2] == 0).all()


@pytest.mark.parametrize("L", [1, 64, 100, 128, 333])
@pytest.mark.parametrize("dtype", DT)
def test_infinite_decay_keeps_nothing(cf, dtype, L):
    """a = 0: y = sigmoid(i) x, and each token's gradients are its own; at any length, the state that is left too."""
    g, dt, C = gen(63), DT[dtype], 40
    x, r, i, dy = (normal(g, 2, L, C, dtype=dt) for _ in range(4))
    decay, h0, dh_last = torch.full((C,), float("inf")), normal(g, 2, C), normal(g, 2, C)
    decay[1::3] = torch.finfo(torch.float32).max
    big = torch.full((C,), 1e30)  # a = 0 in 64 bits too
    y, last, grads, bound = reference(x, r, i, big, h0, None, dy, dh_last)
    gy, gl, gg = both_passes(cf, x, r, i, decay, h0, None, dy, dh_last)
    units = lambda v: R.U * (R.sigmoid_units(v.double()) + 4)  # noqa: E731
    ok(gy, y, y.abs() * units(i), dt, "y")
    ok(gl, last, last.abs() * units(i[:, -1]), torch.float32, "h_last")
    ok(gg["x"], grads["x"], grads["x"].abs() * units(i), dt, "dx")
    s = torch.sigmoid(i.double())
    G = dy.double().clone()
    G[:, -1] += dh_last
    ok(gg["i"], grads["i"], R.U * (G * x.double() * s).abs() * ((R.sigmoid_units(i.double()) + 6) * (1 + s)), dt, "di")
    for k in ("r", "decay", "h0"):
        assert (gg[k] == 0).all() and (grads[k] == 0).all(), k
    pool = h0.cuda()
    z = cf.gated_scan_step(x[:, 0].cuda(), r[:, 0].cuda(), i[:, 0].cuda(), decay.cuda(), pool)
    ok(z, y[:, 0], (y.abs() * units(i))[:, 0], dt, "step")

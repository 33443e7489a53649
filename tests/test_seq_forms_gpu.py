"""Forms of the sequence operators' calls that stand alone: a state or its gradient without the other, checkpoints that
are views, mixtures of checkpoints and tensors, the same tensor twice."""
from __future__ import annotations

import pytest
import torch

import tests.seq_ref as R
import tests.test_seq_gpu as S
from tests.test_seq_gpu import cf  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("given", ["state", "dstate_out"])
@pytest.mark.parametrize("case", [(2, 37, 64, 4, True, True, True, None), (2, 2, 33, 5, False, True, False, None),
                                  (7, 101, 64, 4, True, True, True, "ragged"), (9, 67, 33, 8, True, True, True, "ragged")], ids=str)
@pytest.mark.parametrize("dtype", S.DT)
def test_convolution_with_one_of_state_and_its_gradient(cf, dtype, case, given):  # noqa: F811
    v = S.conv_inputs(case, dtype, seed=71)
    v["dstate_out" if given == "state" else "state"] = None
    ref, z, size = S.conv_grads_ref(v, case[4])
    bounds = S.conv_grad_bounds(v, case[4], z, size)
    d = {k: S.cuda(t) for k, t in v.items()}
    got = cf.conv_causal_grad(d["x"], d["w"], d["dy"], d["bias"], activation="silu" if case[4] else None, state=d["state"],
                              dstate_out=d["dstate_out"], cu_seqlens=d["cu"])
    for k, t in zip(("x", "w", "bias", "state"), got):
        if k not in ref:
            assert t is None
        else:
            S.ok(t, ref[k], bounds[k], S.DT[dtype], "d" + k)


@pytest.mark.parametrize("given", ["h0", "dh_last"])
@pytest.mark.parametrize("case", [(2, 65, 65, True, None), (1, 300, 96, True, None), (9, 203, 64, True, "ragged"),
                                  (5, 97, 32, True, "empty ends")], ids=str)
@pytest.mark.parametrize("dtype", S.DT)
def test_recurrence_with_one_of_state_and_its_gradient(cf, dtype, case, given):  # noqa: F811
    v = S.scan_inputs(case, dtype, seed=72)
    v["decay"] = v["decay"].clamp(min=1e-3)
    v["dh_last" if given == "h0" else "h0"] = None
    ref = S.scan_grads_ref(v)
    args = tuple(S.D(v[k]) for k in ("x", "r", "i", "decay", "h0")) + (v["cu"],)
    bound = R.scan_bounds(*args, S.D(v["dy"]), S.D(v["dh_last"]))
    d = {k: S.cuda(t) for k, t in v.items()}
    states = R.states_of(R.gated_scan(*args)[0], v["cu"]).float().cuda()
    got = cf.gated_scan_grad(d["x"], d["r"], d["i"], d["decay"], d["dy"], states, h0=d["h0"], dh_last=d["dh_last"], cu_seqlens=d["cu"])
    for k, t in zip(("x", "r", "i", "decay", "h0"), got):
        if k not in ref:
            assert t is None
        else:
            kind = torch.float32 if k in ("decay", "h0") else S.DT[dtype]
            S.ok(t, ref[k], bound["d" + k], kind, "d" + k)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype", S.DT)
def test_checkpoints_that_are_views_or_mixed(cf, dtype, packed):  # noqa: F811
    """Checkpoints whose values are slices of wider rows, or beside tensors, are what they stand for, bit for bit."""
    g, dt, C = S.gen(73), S.DT[dtype], 96
    shape = (150, C) if packed else (2, 75, C)
    cu = torch.tensor([0, 40, 41, 120], dtype=torch.int32).cuda() if packed else None
    x, r, i, dy = (S.normal(g, *shape, dtype=dt).cuda() for _ in range(4))
    w, b, decay = S.normal(g, C, 4, dtype=dt).cuda(), S.normal(g, C, dtype=dt).cuda(), torch.exp(torch.rand(C, generator=g) * 5 - 5).cuda()
    p = {k: cf.act8_pack(t) for k, t in dict(x=x, r=r, i=i).items()}
    whole = {k: cf.act8_unpack(t) for k, t in p.items()}

    def view(a, at):
        wide = torch.zeros(*a.shape[:-1], a.shape[-1] + 64, dtype=a.dtype, device="cuda")
        wide[..., at : at + a.shape[-1]] = a
        return wide[..., at : at + a.shape[-1]]

    states = cf.gated_scan(whole["x"], whole["r"], whole["i"], decay, cu_seqlens=cu, save_states=True)[2]
    ref = cf.gated_scan_grad(p["x"], p["r"], p["i"], decay, dy, states, cu_seqlens=cu)
    cref = cf.conv_causal_grad(p["x"], w, dy, b, activation="silu", cu_seqlens=cu)
    for at in (32, 7):
        q = {k: cf.Act8(view(t.q, at), view(t.scale, 3), t.dtype) for k, t in p.items()}
        assert torch.equal(cf.act8_unpack(q["x"]), whole["x"])
        got = cf.gated_scan_grad(q["x"], q["r"], q["i"], decay, view(dy, at), states, cu_seqlens=cu)
        close = lambda a, c: torch.allclose(a.float(), c.float(), rtol=2 * torch.finfo(a.dtype).eps, atol=1e-4)  # noqa: E731
        assert all(close(a, c) for a, c in zip(got[:4], ref[:4]))
        got = cf.conv_causal_grad(q["x"], w, view(dy, at), b, activation="silu", cu_seqlens=cu)
        assert all(close(a, c) for a, c in zip(got[:3], cref[:3]))
    plain = cf.gated_scan_grad(whole["x"], whole["r"], whole["i"], decay, dy, states, cu_seqlens=cu)
    for mix in ((p["x"], whole["r"], whole["i"]), (whole["x"], p["r"], p["i"]), (p["x"], p["r"], whole["i"])):
        got = cf.gated_scan_grad(*mix, decay, dy, states, cu_seqlens=cu)
        assert all(torch.equal(a, c) for a, c in zip(got[:4], plain[:4]))


def test_one_tensor_as_several_inputs(cf):  # noqa: F811
    """x, r, i and dy may be one tensor, and rows one row (stride 0), as a sum's gradient has them."""
    g = S.gen(74)
    x = S.normal(g, 2, 90, 40, dtype=torch.float32).cuda()
    decay, w = torch.rand(40, generator=g).cuda(), S.normal(g, 40, 4, dtype=torch.float32).cuda()
    y, last, states = cf.gated_scan(x, x, x, decay, save_states=True)
    yc, lc, sc = cf.gated_scan(x, x.clone(), x.clone(), decay, save_states=True)
    assert torch.equal(y, yc) and torch.equal(last, lc) and torch.equal(states, sc)
    one = torch.ones((), device="cuda").expand(2, 90, 40)
    for dy in (x, one):
        for a, c in zip(cf.gated_scan_grad(x, x, x, decay, dy, states)[:4], cf.gated_scan_grad(x, x.clone(), x.clone(), decay, dy.clone().contiguous(), states)):
            assert torch.equal(a, c)
        for a, c in zip(cf.conv_causal_grad(x, w, dy)[:2], cf.conv_causal_grad(x, w, dy.clone().contiguous())):
            assert torch.equal(a, c)
    z = x[0, :5].contiguous()
    h, k = torch.zeros(5, 40, device="cuda"), torch.zeros(5, 40, device="cuda")
    assert torch.equal(cf.gated_scan_step(z, z, z, decay, h), cf.gated_scan_step(z, z.clone(), z.clone(), decay, k)) and torch.equal(h, k)

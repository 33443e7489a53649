"""The sequence operators against their plain 64-bit forms, on the GPU."""
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


def normal(g, *shape, dtype, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def offsets(g, kind, rows, n):
    """cu_seqlens: some empty, some of one token, the last before the end of the rows."""
    if kind == "ragged":
        cut = torch.sort(torch.randint(0, rows - rows // 10 + 1, (n - 1,), generator=g)).values
        if n > 4:
            cut[1] = cut[0]
            cut[3] = torch.minimum(cut[2] + 1, cut[3])
        return torch.cat([torch.zeros(1, dtype=torch.long), cut, torch.tensor([rows - rows // 10])]).int()
    if kind == "empty ends":  # empty sequences first and last, no unused rows
        return torch.tensor([0, 0, rows // 3, rows // 3, rows, rows], dtype=torch.int32)
    if kind == "none used":
        return torch.zeros(n + 1, dtype=torch.int32)
    raise ValueError(kind)


def cuda(t):
    return t.cuda() if isinstance(t, torch.Tensor) else t


def D(t):
    return None if t is None else t.double()


def ok(got, ref, bound, dtype, name):
    w = R.worst(got, ref, bound, dtype)
    assert w <= 1.0, f"{name}: {w:.3g} times what rounding allows"


# ---- 8-bit checkpoints --------------------------------------------------


def hard_rows(g, C, dtype):
    """Rows with what goes wrong: zeros, halves, the type's ends, subnormals, infinities and NaN."""
    f = torch.finfo(dtype)
    x = normal(g, 12, C, dtype=dtype)
    x[0] = 0
    x[1] = (torch.arange(C) % 31 - 15).to(dtype) / 2 + 0.5  # ties at every step
    x[2, ::3] = f.max
    x[3] = (x[3] * 100).to(dtype) * f.smallest_normal
    x[4, C // 2] = float("inf")
    x[5, -1] = float("nan")
    x[6] = 127.0
    x[7] = 128.0
    x[8] = -127.5 if dtype != torch.bfloat16 else -127.0
    x[9, 1:] = 0
    x[10] = f.smallest_normal * f.eps
    return x


@pytest.mark.parametrize("C", [1, 8, 31, 32, 40, 65, 256, 1000])
@pytest.mark.parametrize("dtype", DT)
def test_act8_is_its_definition(cf, dtype, C):
    g = gen(C)
    x = torch.cat([normal(g, 37, C, dtype=DT[dtype]) * 2 ** torch.randint(-8, 9, (37, 1), generator=g).to(DT[dtype]),
                   hard_rows(g, C, DT[dtype])])
    q, scale = R.act8(x)
    p = cf.act8_pack(x.cuda())
    assert torch.equal(p.scale.cpu(), scale) and torch.equal(p.q.cpu(), q)
    back = cf.act8_unpack(p)
    assert back.dtype == DT[dtype]
    ref = R.act8_values(q, scale)
    assert torch.equal(back.cpu().double().nan_to_num(nan=1e300), ref.nan_to_num(nan=1e300))
    fine = torch.isfinite(ref)
    step = torch.exp2(scale.double() - 127).repeat_interleave(32, -1)[:, :C]
    top = x.double().abs() > 63.5 * step  # where the type's end stops the rounding
    assert ((x.double() - ref).abs() <= torch.where(top, step, step / 2))[fine].all()


@pytest.mark.parametrize("dtype", DT)
def test_act8_takes_strided_rows_any_rank_and_unaligned_memory(cf, dtype):
    g = gen(3)
    wide = normal(g, 20, 200, dtype=DT[dtype]).cuda()
    for x in (wide[:, 40:136], wide[:, 3:100], wide[::2, :64], wide.view(4, 5, 200), wide.t(), wide[0]):
        q, scale = R.act8(x.cpu())
        p = cf.act8_pack(x)
        assert p.q.shape == x.shape and torch.equal(p.q.cpu(), q) and torch.equal(p.scale.cpu(), scale)
        assert torch.equal(cf.act8_unpack(p).cpu().double(), R.act8_values(q, scale))
    out = torch.empty(20 * 200 + 1, dtype=DT[dtype], device="cuda")[1:].view(20, 200)
    p = cf.act8_pack(wide)
    assert torch.equal(cf.act8_unpack(p, out=out), cf.act8_unpack(p)) and out.data_ptr() % 16 != 0
    assert cf.act8_pack(wide[:0]).q.shape == (0, 200)


@pytest.mark.parametrize("geometry", [(2, 12, 11, 32, 48), (2, 12, 11, 64, 256)])
def test_weight_gradient_from_a_checkpoint(cf, geometry):
    """conv_wgrad of the checkpoint is conv_wgrad of what it stands for, bit for bit."""
    N, H, W, C, O = geometry
    g = gen(7)
    x, dy = normal(g, N, H, W, C, dtype=torch.bfloat16).cuda(), normal(g, N, H, W, O, dtype=torch.bfloat16).cuda()
    p = cf.act8_pack(x)
    got = cf.conv_wgrad(p, dy, 3, padding=1)
    assert torch.equal(got, cf.conv_wgrad(cf.act8_unpack(p), dy, 3, padding=1))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = cf.conv_wgrad(p, dy, (3, 3), padding=1, stream=side)
    side.synchronize()
    assert torch.equal(got, other)
    assert not torch.equal(got, cf.conv_wgrad(x, dy, 3, padding=1))
    with pytest.raises(TypeError):
        cf.conv_wgrad(p, dy.half(), 3, padding=1)


# ---- causal convolution -------------------------------------------------

CONV = [  # (n, L, C, K, silu, state, bias, packed)
    (1, 1, 1, 1, False, False, False, None),
    (2, 1, 8, 4, True, True, True, None),
    (3, 2, 20, 4, False, True, True, None),
    (2, 37, 64, 4, True, False, True, None),
    (2, 70, 65, 3, True, True, True, None),
    (1, 131, 96, 2, False, False, False, None),
    (2, 50, 40, 5, True, True, False, None),
    (2, 45, 24, 8, True, True, True, None),
    (3, 0, 16, 4, True, True, True, None),
    (7, 101, 64, 4, True, True, True, "ragged"),
    (9, 67, 33, 3, False, True, True, "ragged"),
    (7, 90, 16, 7, True, False, True, "ragged"),
    (5, 61, 32, 4, True, True, True, "empty ends"),
    (3, 9, 16, 4, True, True, True, "none used"),
]


def conv_inputs(case, dtype, seed=0):
    n, L, C, K, silu, has_state, has_bias, packed = case
    g, dt = gen(seed), DT[dtype]
    cu = offsets(g, packed, L, n) if packed else None
    n = len(cu) - 1 if packed else n
    shape = (L, C) if packed else (n, L, C)
    return dict(x=normal(g, *shape, dtype=dt), w=normal(g, C, K, dtype=dt, scale=K ** -0.5),
                bias=normal(g, C, dtype=dt, scale=0.3) if has_bias else None,
                state=normal(g, n, K - 1, C, dtype=dt) if has_state else None, cu=cu,
                dy=normal(g, *shape, dtype=dt), dstate_out=normal(g, n, K - 1, C, dtype=dt) if has_state else None)


@pytest.mark.parametrize("case", CONV, ids=str)
@pytest.mark.parametrize("dtype", DT)
def test_conv_causal(cf, dtype, case):
    silu, K = case[4], case[3]
    v = conv_inputs(case, dtype)
    y, left, z, S = R.conv_causal(D(v["x"]), D(v["w"]), D(v["bias"]), silu, D(v["state"]), v["cu"])
    d = {k: cuda(t) for k, t in v.items()}
    got, state = cf.conv_causal(d["x"], d["w"], d["bias"], activation="silu" if silu else None, state=d["state"],
                                cu_seqlens=d["cu"], return_state=True)
    ok(got, y, R.conv_bound(z, S, K, silu), DT[dtype], "y")
    assert torch.equal(state.cpu().double(), left)
    # a given output: the same, but for unused rows, which stay
    out = torch.full_like(got, 7.0)
    assert cf.conv_causal(d["x"], d["w"], d["bias"], activation="silu" if silu else None, state=d["state"],
                          cu_seqlens=d["cu"], out=out) is out
    used = int(v["cu"][-1]) if v["cu"] is not None else None
    if used is None:
        assert torch.equal(out, got)
    else:
        assert torch.equal(out[:used], got[:used]) and (out[used:] == 7).all() and (got[used:] == 0).all()


def conv_grads_ref(v, silu):
    t = {k: (D(a).requires_grad_() if k in ("x", "w", "bias", "state") and a is not None else a) for k, a in v.items()}
    y, left, z, S = R.conv_causal(t["x"], t["w"], t["bias"], silu, t["state"], v["cu"])
    loss = (y * D(v["dy"])).sum()
    if v["dstate_out"] is not None:
        loss = loss + (left * D(v["dstate_out"])).sum()
    names = [k for k in ("x", "w", "bias", "state") if t[k] is not None]
    grads = torch.autograd.grad(loss, [t[k] for k in names], allow_unused=True)
    return {k: (torch.zeros_like(t[k]) if q is None else q) for k, q in zip(names, grads)}, z.detach(), S.detach()


def conv_grad_bounds(v, silu, z, S):
    """Bounds of dx, dw, dbias, dstate: the slope's error and one unit a product, through the same sums on magnitudes."""
    K = v["w"].shape[1]
    m = {k: (D(a).abs() if isinstance(a, torch.Tensor) and k != "cu" else a) for k, a in v.items()}
    s = torch.sigmoid(z)
    # the largest |dz| and what it is off by
    slope = (s * (1 + z.abs() * (1 - s))) if silu else torch.ones_like(z)
    dz = m["dy"] * slope
    bz = (m["dy"] * R.slope_bound(z, S, K) if silu else 0 * dz) + R.U * dz
    used = torch.zeros_like(dz)
    cu = v["cu"]
    X = dict(x=m["x"].requires_grad_(), w=m["w"].requires_grad_())
    b = torch.zeros(m["w"].shape[0], dtype=torch.float64, requires_grad=True)
    st = m["state"].requires_grad_() if m["state"] is not None else None
    y, left, _, _ = R.conv_causal(X["x"], X["w"], b, False, st, cu)
    leaves = [X["x"], X["w"], b] + ([st] if st is not None else [])
    out = {}
    for what, weight in (("off", bz), ("size", dz)):
        loss = (y * weight).sum()
        if m["dstate_out"] is not None:
            loss = loss + (left * m["dstate_out"]).sum() * (1 if what == "size" else 0)
        gs = torch.autograd.grad(loss, leaves, retain_graph=True, allow_unused=True)
        out[what] = [torch.zeros_like(t) if q is None else q for t, q in zip(leaves, gs)]
    names = ["x", "w", "bias"] + (["state"] if st is not None else [])
    chain = {"x": K + 2, "state": K + 2, "w": 512, "bias": 512}  # additions one after the other
    return {k: out["off"][j] + R.U * (chain[k] + 2) * out["size"][j] for j, k in enumerate(names)}


@pytest.mark.parametrize("saved8", [False, True], ids=["", "8bit"])
@pytest.mark.parametrize("case", CONV, ids=str)
@pytest.mark.parametrize("dtype", DT)
def test_conv_causal_grad(cf, dtype, case, saved8):
    silu = case[4]
    v = conv_inputs(case, dtype, seed=1)
    x = v["x"].cuda()
    if saved8:
        q, scale = R.act8(v["x"])
        x = cf.Act8(q.cuda(), scale.cuda(), DT[dtype])
        v["x"] = R.act8_values(q, scale)
    ref, z, S = conv_grads_ref(v, silu)
    bounds = conv_grad_bounds(v, silu, z, S)
    d = {k: cuda(t) for k, t in v.items()}
    got = cf.conv_causal_grad(x, d["w"], d["dy"], d["bias"], activation="silu" if silu else None, state=d["state"],
                              dstate_out=d["dstate_out"], cu_seqlens=d["cu"])
    for k, t in zip(("x", "w", "bias", "state"), got):
        if k not in ref:
            assert t is None
            continue
        assert t.dtype == DT[dtype]
        ok(t, ref[k], bounds[k], DT[dtype], "d" + k)
    again = cf.conv_causal_grad(x, d["w"], d["dy"], d["bias"], activation="silu" if silu else None, state=d["state"],
                                dstate_out=d["dstate_out"], cu_seqlens=d["cu"])
    assert all(a is b or torch.equal(a, b) for a, b in zip(got, again))


def test_conv_causal_continues_from_its_state(cf):
    """A sequence in pieces, each from the window the one before left, is the sequence in one."""
    g = gen(5)
    for dtype in DT.values():
        x, w, b = normal(g, 2, 57, 48, dtype=dtype).cuda(), normal(g, 48, 4, dtype=dtype).cuda(), normal(g, 48, dtype=dtype).cuda()
        whole, end = cf.conv_causal(x, w, b, activation="silu", return_state=True)
        state, parts = None, []
        for lo, hi in ((0, 1), (1, 3), (3, 20), (20, 20), (20, 57)):
            y, state = cf.conv_causal(x[:, lo:hi], w, b, activation="silu", state=state, return_state=True)
            parts.append(y)
        assert torch.equal(torch.cat(parts, 1), whole) and torch.equal(state, end)


@pytest.mark.parametrize("K,C", [(1, 24), (2, 33), (3, 64), (4, 64), (4, 1), (6, 40), (8, 2000)])
@pytest.mark.parametrize("dtype", DT)
def test_conv_causal_step(cf, dtype, K, C):
    """Token by token is the whole sequence; skipped rows, slots of other requests and repeated slots."""
    g, dt = gen(K), DT[dtype]
    B, T, slots = 5, 6, 9
    x, w, b = normal(g, B, T, C, dtype=dt).cuda(), normal(g, C, K, dtype=dt).cuda(), normal(g, C, dtype=dt).cuda()
    start = normal(g, slots, K - 1, C, dtype=dt).cuda()
    index = torch.tensor([7, 0, -1, 3, slots], dtype=torch.int32).cuda()
    rows = torch.tensor([0, 1, 3]).cuda()
    whole, end = cf.conv_causal(x[rows], w, b, activation="silu", state=start[index[rows].long()], return_state=True)
    pool = start.clone()
    for t in range(T):
        y = cf.conv_causal_step(x[:, t], w, pool, b, activation="silu", index=index)
        assert torch.equal(y[rows], whole[:, t]) and (y[[2, 4]] == 0).all()
    assert torch.equal(pool[index[rows].long()], end)
    idle = torch.tensor([k for k in range(slots) if k not in (7, 0, 3)]).cuda()
    assert torch.equal(pool[idle], start[idle])
    # without an index: the first rows of the pool; out given
    pool, out = start[:B].clone(), torch.full((B, C), 5.0, dtype=dt, device="cuda")
    y = cf.conv_causal_step(x[:, 0], w, pool, b, index=None, out=out)
    ref = cf.conv_causal(x[:, :1], w, b, state=start[:B])[:, 0]
    assert y is out and torch.equal(y, ref)
    out.fill_(5.0)
    cf.conv_causal_step(x[:, 0], w, start.clone(), b, index=index, out=out)
    assert (out[[2, 4]] == 5).all()
    # one slot named by all rows: its tokens in order
    pool, many = start.clone(), x.reshape(-1, C)
    y = cf.conv_causal_step(many, w, pool, b, index=torch.full((many.shape[0],), 4, dtype=torch.int32).cuda())
    ref, end = cf.conv_causal(many[None], w, b, state=start[4:5], return_state=True)
    assert torch.equal(y, ref[0]) and torch.equal(pool[4], end[0])
    two = torch.tensor([1, 2] * 40, dtype=torch.int32).cuda()
    big, pool = normal(g, 80, C, dtype=dt).cuda(), start.clone()
    y = cf.conv_causal_step(big, w, pool, b, index=two)
    ref = cf.conv_causal(torch.stack([big[::2], big[1::2]]), w, b, state=start[1:3])
    assert torch.equal(y[::2], ref[0]) and torch.equal(y[1::2], ref[1])


# ---- gated recurrence ---------------------------------------------------

SCAN = [  # (n, L, C, h0, packed)
    (1, 1, 1, False, None),
    (3, 1, 24, True, None),
    (2, 63, 64, False, None),
    (2, 65, 65, True, None),
    (1, 300, 96, True, None),
    (2, 517, 40, False, None),
    (1, 1300, 8, True, None),
    (2, 0, 16, True, None),
    (9, 203, 64, True, "ragged"),
    (12, 701, 33, True, "ragged"),
    (6, 330, 130, False, "ragged"),
    (5, 97, 32, True, "empty ends"),
    (3, 70, 16, True, "none used"),
]


def scan_inputs(case, dtype, seed=0):
    n, L, C, has_h0, packed = case
    g, dt = gen(seed), DT[dtype]
    cu = offsets(g, packed, L, n) if packed else None
    n = len(cu) - 1 if packed else n
    shape = (L, C) if packed else (n, L, C)
    # slow and fast channels, one with a = 1
    decay = torch.exp(torch.rand(C, generator=g) * 9 - 7)
    decay[C // 2] = 0
    v = dict(x=normal(g, *shape, dtype=dt), r=normal(g, *shape, dtype=dt, scale=2), i=normal(g, *shape, dtype=dt, scale=2),
             decay=decay, h0=normal(g, n, C, dtype=torch.float32) if has_h0 else None, cu=cu, dy=normal(g, *shape, dtype=dt),
             dh_last=normal(g, n, C, dtype=torch.float32) if has_h0 else None)
    return v


@pytest.mark.parametrize("case", SCAN, ids=str)
@pytest.mark.parametrize("dtype", DT)
def test_gated_scan(cf, dtype, case):
    v = scan_inputs(case, dtype)
    args = (D(v["x"]), D(v["r"]), D(v["i"]), D(v["decay"]), D(v["h0"]), v["cu"])
    y, last = R.gated_scan(*args)
    bound = R.scan_bounds(*args)
    d = {k: cuda(t) for k, t in v.items()}
    got, end, states = cf.gated_scan(d["x"], d["r"], d["i"], d["decay"], h0=d["h0"], cu_seqlens=d["cu"], save_states=True)
    ok(got, y, bound["y"], DT[dtype], "y")
    ok(end, last, bound["last"], torch.float32, "h_last")
    assert torch.isfinite(states).all() and states.dtype == torch.float32
    ref, lim = R.states_of(y, v["cu"]), R.states_of(bound["y"], v["cu"])
    inner = torch.tensor([k for k in range(ref.shape[1]) if v["cu"] is None and k > 0 or v["cu"] is not None and any(
        lo < 64 * k < hi for _, lo, hi in R.ranges(0, 0, v["cu"]))], dtype=torch.long)
    ok(states[:, inner.cuda()], ref[:, inner], lim[:, inner], torch.float32, "states")
    out = torch.full_like(got, 7.0)
    again, end2 = cf.gated_scan(d["x"], d["r"], d["i"], d["decay"], h0=d["h0"], cu_seqlens=d["cu"], out=out)
    assert again is out and torch.equal(end, end2)
    used = int(v["cu"][-1]) if v["cu"] is not None else None
    if used is None:
        assert torch.equal(out, got)
    else:
        assert torch.equal(out[:used], got[:used]) and (out[used:] == 7).all() and (got[used:] == 0).all()


def scan_grads_ref(v):
    t = {k: (D(a).requires_grad_() if k in ("x", "r", "i", "decay", "h0") and a is not None else a) for k, a in v.items()}
    y, last = R.gated_scan(t["x"], t["r"], t["i"], t["decay"], t["h0"], v["cu"])
    loss = (y * D(v["dy"])).sum()
    if v["dh_last"] is not None:
        loss = loss + (last * D(v["dh_last"])).sum()
    names = [k for k in ("x", "r", "i", "decay", "h0") if t[k] is not None]
    grads = torch.autograd.grad(loss, [t[k] for k in names], allow_unused=True) if loss.requires_grad else [None] * len(names)
    return {k: (torch.zeros_like(t[k]) if q is None else q) for k, q in zip(names, grads)}


@pytest.mark.parametrize("saved8", [False, True], ids=["", "8bit"])
@pytest.mark.parametrize("case", SCAN, ids=str)
@pytest.mark.parametrize("dtype", DT)
def test_gated_scan_grad(cf, dtype, case, saved8):
    v = scan_inputs(case, dtype, seed=1)
    v["decay"] = v["decay"].clamp(min=1e-3)  # a = 1 has no derivative (its own test below)
    saved = {k: v[k].cuda() for k in ("x", "r", "i")}
    if saved8:
        for k in saved:
            q, scale = R.act8(v[k])
            saved[k] = cf.Act8(q.cuda(), scale.cuda(), DT[dtype])
            v[k] = R.act8_values(q, scale)
    ref = scan_grads_ref(v)
    args = (D(v["x"]), D(v["r"]), D(v["i"]), D(v["decay"]), D(v["h0"]), v["cu"])
    bound = R.scan_bounds(*args, D(v["dy"]), D(v["dh_last"]))
    d = {k: cuda(t) for k, t in v.items()}
    states = R.states_of(R.gated_scan(*args)[0], v["cu"]).float().cuda()
    call = dict(h0=d["h0"], dh_last=d["dh_last"], cu_seqlens=d["cu"])
    got = cf.gated_scan_grad(saved["x"], saved["r"], saved["i"], d["decay"], d["dy"], states, **call)
    for k, t in zip(("x", "r", "i", "decay", "h0"), got):
        if k not in ref:
            assert t is None
            continue
        kind = torch.float32 if k in ("decay", "h0") else DT[dtype]
        assert t.dtype == kind
        ok(t, ref[k], bound["d" + k], kind, "d" + k)
    again = cf.gated_scan_grad(saved["x"], saved["r"], saved["i"], d["decay"], d["dy"], states, **call)
    assert all(a is b or torch.equal(a, b) for a, b in zip(got, again))


def test_gated_scan_gates_at_their_ends(cf):
    """Gates of +-infinity and 0 decay: a = 1 keeps the state and takes nothing in, with finite gradients."""
    for dtype in DT.values():
        g = gen(2)
        x, r, i = (normal(g, 1, 70, 8, dtype=dtype) for _ in range(3))
        decay = torch.full((8,), 0.5)
        decay[1] = 0
        r[:, :, 2] = float("-inf")
        r[:, :, 3] = float("inf")
        i[:, :, 4] = float("-inf")
        i[:, :, 5] = float("inf")
        decay[6] = 200.0
        h0 = torch.ones(1, 8)
        y, last = R.gated_scan(D(x), D(r), D(i), D(decay), D(h0), None)
        d = [t.cuda() for t in (x, r, i, decay)]
        got, end, states = cf.gated_scan(*d, h0=h0.cuda(), save_states=True)
        fine = torch.tensor([0, 1, 2, 3, 4, 5, 6, 7])
        lim = R.scan_bounds(D(x), D(r.clamp(-60, 60)), D(i.clamp(-60, 60)), D(decay), D(h0), None)
        ok(got[..., fine], y[..., fine], lim["y"][..., fine].nan_to_num() + 1e-12, dtype, "y")
        assert (got[..., 1:3] == 1).all() and (end[:, 1:3] == 1).all()
        grads = cf.gated_scan_grad(*d, torch.ones_like(d[0]), states, h0=h0.cuda())
        for t in grads:
            assert torch.isfinite(t).all()
        assert (grads[1][..., 1:3] == 0).all() and (grads[0][..., 1:3] == 0).all() and (grads[4][:, 1] == 70).all()
        # r = inf: s is a reciprocal (1 ulp) times its own argument (half an ulp), so 1 - s is at most 2^-22, and
        # |dr| = decay |dl| s (1 - s) with |dl| <= a |G| (|h| + a g |x| / m): a = e^-1/2, m = 0.795, |G| <= 1 / (1 - a)
        # = 2.54, |g x| <= 5, |h| <= |h0| + m |g x| / (1 - a) <= 11.1: |dl| <= 0.607 * 2.54 * (11.1 + 3.9) = 23.2
        assert x.abs().max() <= 5 and (grads[1][..., 3].float().abs() <= 0.5 * 23.2 * 2 ** -22).all()


def test_gated_scan_continues_from_its_state(cf):
    g = gen(6)
    for dtype in DT.values():
        x, r, i = (normal(g, 2, 300, 40, dtype=dtype) for _ in range(3))
        decay = torch.exp(torch.rand(40, generator=g) * 9 - 7)
        bound = R.scan_bounds(D(x), D(r), D(i), D(decay), None, None)
        ref, last = R.gated_scan(D(x), D(r), D(i), D(decay), None, None)
        x, r, i, decay = (t.cuda() for t in (x, r, i, decay))
        state, parts = None, []
        for lo, hi in ((0, 1), (1, 80), (80, 80), (80, 293)):
            y, state = cf.gated_scan(x[:, lo:hi], r[:, lo:hi], i[:, lo:hi], decay, h0=state)
            parts.append(y)
        for t in range(293, 300):
            parts.append(cf.gated_scan_step(x[:, t], r[:, t], i[:, t], decay, state)[:, None])
        ok(torch.cat(parts, 1), ref, bound["y"], dtype, "y")
        ok(state, last, bound["last"], torch.float32, "state")


@pytest.mark.parametrize("C", [1, 33, 64, 2000])
@pytest.mark.parametrize("dtype", DT)
def test_gated_scan_step(cf, dtype, C):
    g, dt = gen(C), DT[dtype]
    B, slots = 5, 9
    x, r, i = (normal(g, B, C, dtype=dt) for _ in range(3))
    decay, start = torch.exp(torch.rand(C, generator=g) * 9 - 7), normal(g, slots, C, dtype=torch.float32)
    index = torch.tensor([7, 0, -1, 3, slots], dtype=torch.int32)
    rows = torch.tensor([0, 1, 3])
    at = index[rows].long()
    args = (D(x[rows, None]), D(r[rows, None]), D(i[rows, None]), D(decay), D(start[at]), None)
    ref, last = R.gated_scan(*args)
    bound = R.scan_bounds(*args)
    d = [t.cuda() for t in (x, r, i, decay)]
    pool = start.cuda()
    y = cf.gated_scan_step(*d, pool, index=index.cuda())
    ok(y[rows.cuda()], ref[:, 0], bound["y"][:, 0], dt, "y")
    ok(pool[at.cuda()], last, bound["last"], torch.float32, "h")
    assert (y[[2, 4]] == 0).all()
    idle = [k for k in range(slots) if k not in (7, 0, 3)]
    assert torch.equal(pool[idle].cpu(), start[idle])
    out = torch.full((B, C), 5.0, dtype=dt, device="cuda")
    assert cf.gated_scan_step(*d, start.cuda(), index=index.cuda(), out=out) is out
    assert (out[[2, 4]] == 5).all() and torch.equal(out[[0, 1, 3]], y[[0, 1, 3]])
    # one slot named by every row, and two in turn: their tokens in order
    for idx in ([4] * B, [1, 2, 1, 1, 2]):
        pool = start.cuda()
        y = cf.gated_scan_step(*d, pool, index=torch.tensor(idx, dtype=torch.int32).cuda())
        for slot in set(idx):
            k = [j for j in range(B) if idx[j] == slot]
            a = (D(x[None, k]), D(r[None, k]), D(i[None, k]), D(decay), D(start[slot][None]), None)
            ref, last = R.gated_scan(*a)
            lim = R.scan_bounds(*a)
            ok(y[k], ref[0], lim["y"][0], dt, "y")
            ok(pool[slot][None], last, lim["last"], torch.float32, "h")


# ---- memory, streams, graphs --------------------------------------------


@pytest.mark.parametrize("dtype", DT)
def test_strided_and_unaligned_inputs_are_their_contiguous_copies(cf, dtype):
    g, dt = gen(8), DT[dtype]
    N, L, C = 2, 75, 64
    wide = normal(g, N, L + 3, 4 * C + 9, dtype=dt).cuda()
    decay = torch.exp(torch.rand(C, generator=g) * 9 - 7).cuda()
    w, b = normal(g, C, 4, dtype=dt).cuda(), normal(g, C, dtype=dt).cuda()
    views = {
        "fused": [wide[:, :L, k * C : (k + 1) * C] for k in range(4)],
        "odd offset": [wide[:, 1 : L + 1, k * C + 3 : (k + 1) * C + 3] for k in range(4)],
        "token stride 0": [wide[:, :1, k * C : (k + 1) * C].expand(N, L, C) for k in range(4)],
        "batch stride 0": [wide[:1, :L, k * C : (k + 1) * C].expand(N, L, C) for k in range(4)],
        "transposed": [wide[:, :L, k * C : (k + 1) * C].transpose(1, 2).contiguous().transpose(1, 2) for k in range(4)],
    }
    for name, (x, r, i, dy) in views.items():
        cx, cr, ci, cy = (t.contiguous() for t in (x, r, i, dy))
        y, last, states = cf.gated_scan(x, r, i, decay, save_states=True)
        yc, lc, sc = cf.gated_scan(cx, cr, ci, decay, save_states=True)
        for a, q in ((y, yc), (last, lc), (states, sc)):
            assert torch.allclose(a.float(), q.float(), rtol=1e-2 if dtype != "f32" else 1e-5, atol=1e-5), name
        for a, q in zip(cf.gated_scan_grad(x, r, i, decay, dy, sc)[:4], cf.gated_scan_grad(cx, cr, ci, decay, cy, sc)[:4]):
            assert torch.allclose(a.float(), q.float(), rtol=1e-2 if dtype != "f32" else 1e-4, atol=1e-4), name
        assert torch.equal(cf.conv_causal(x, w, b, activation="silu"), cf.conv_causal(cx, w, b, activation="silu")), name
        for a, q in zip(cf.conv_causal_grad(x, w, dy, b)[:3], cf.conv_causal_grad(cx, w, cy, b)[:3]):
            assert torch.allclose(a.float(), q.float(), rtol=1e-2 if dtype != "f32" else 1e-4, atol=1e-4), name


def test_nan_stays_in_its_sequence(cf):
    """NaN and infinities in one packed sequence, and in rows of none, reach no other sequence and no sum of them."""
    g = gen(9)
    cu = torch.tensor([0, 100, 130, 260, 400], dtype=torch.int32).cuda()
    rows, C = 450, 64
    for dtype in DT.values():
        x, r, i, dy = (normal(g, rows, C, dtype=dtype).cuda() for _ in range(4))
        decay = torch.exp(torch.rand(C, generator=g) * 9 - 7).cuda()
        w, b = normal(g, C, 4, dtype=dtype).cuda(), normal(g, C, dtype=dtype).cuda()
        clean = [t.clone() for t in (x, r, i, dy)]
        for t in (x, r, i, dy):
            t[105:128:3] = float("nan")
            t[110] = float("inf")
            t[400:] = float("nan")
        keep = torch.cat([torch.arange(100), torch.arange(130, 400)]).cuda()
        y, last, states = cf.gated_scan(x, r, i, decay, cu_seqlens=cu, save_states=True)
        yc, lc, sc = cf.gated_scan(*clean[:3], decay, cu_seqlens=cu, save_states=True)
        assert torch.equal(y[keep], yc[keep]) and torch.equal(last[[0, 2, 3]], lc[[0, 2, 3]]) and (y[400:] == 0).all()
        grads = cf.gated_scan_grad(x, r, i, decay, dy, states, cu_seqlens=cu)
        gc = cf.gated_scan_grad(*clean[:3], decay, clean[3], sc, cu_seqlens=cu)
        for a, q in zip(grads[:3], gc[:3]):
            assert torch.equal(a[keep], q[keep]) and (a[400:] == 0).all()
        z = cf.conv_causal(x, w, b, activation="silu", cu_seqlens=cu)
        assert torch.equal(z[keep], cf.conv_causal(clean[0], w, b, activation="silu", cu_seqlens=cu)[keep])
        dx = cf.conv_causal_grad(x, w, dy, b, activation="silu", cu_seqlens=cu)[0]
        assert torch.equal(dx[keep], cf.conv_causal_grad(clean[0], w, clean[3], b, activation="silu", cu_seqlens=cu)[0][keep])
        # rows of no sequence reach no sum
        clean_tail = [t.clone() for t in clean]
        for t in clean_tail:
            t[400:] = float("nan")
        a = cf.gated_scan_grad(*clean_tail[:3], decay, clean_tail[3], sc, cu_seqlens=cu)
        assert torch.equal(a[3], gc[3])
        a = cf.conv_causal_grad(clean_tail[0], w, clean_tail[3], b, activation="silu", cu_seqlens=cu)
        q = cf.conv_causal_grad(clean[0], w, clean[3], b, activation="silu", cu_seqlens=cu)
        assert torch.equal(a[1], q[1]) and torch.equal(a[2], q[2])


def block(cf, v, stream=None):
    """A recurrent block's training step: forward, its activations in 8 bits, backward from them."""
    kw = dict(cu_seqlens=v["cu"], stream=stream)
    u = cf.conv_causal(v["x"], v["w"], v["b"], activation="silu", **kw)
    y, last, states = cf.gated_scan(u, v["r"], v["i"], v["decay"], save_states=True, **kw)
    x8, u8, r8, i8 = (cf.act8_pack(t, stream=stream) for t in (v["x"], u, v["r"], v["i"]))
    du, dr, di, dd, _ = cf.gated_scan_grad(u8, r8, i8, v["decay"], v["dy"], states, **kw)
    dx, dw, db, _ = cf.conv_causal_grad(x8, v["w"], du, v["b"], activation="silu", **kw)
    return [y, last, dx, dw, db, dr, di, dd]


def block_inputs(seed, rows=333, C=96, dtype=torch.bfloat16):
    g = gen(seed)
    x, r, i, dy = (normal(g, rows, C, dtype=dtype).cuda() for _ in range(4))
    return dict(x=x, r=r, i=i, dy=dy, w=normal(g, C, 4, dtype=dtype, scale=0.5).cuda(), b=normal(g, C, dtype=dtype).cuda(),
                decay=torch.exp(torch.rand(C, generator=g) * 7 - 6).cuda(), cu=offsets(g, "ragged", rows, 8).cuda())


def test_block_together(cf):
    """The operators as a recurrent block runs them, against autograd in 64 bits.  8-bit activations leave each gradient
    within a few per cent: a step of a block of 32 normal values is about 2^-5 of their size, off by 0.3 of that."""
    v = block_inputs(11)
    got = block(cf, v)
    t = {k: (a.cpu().double() if a.is_floating_point() else a.cpu()) for k, a in v.items()}
    for k in ("x", "w", "b", "r", "i", "decay"):
        t[k].requires_grad_()
    u = R.conv_causal(t["x"], t["w"], t["b"], True, None, t["cu"])[0]
    y, last = R.gated_scan(u, t["r"], t["i"], t["decay"], None, t["cu"])
    grads = torch.autograd.grad((y * t["dy"]).sum(), [t[k] for k in ("x", "w", "b", "r", "i", "decay")])
    far = lambda a, b: float((a.cpu().double() - b).norm() / b.norm())  # noqa: E731
    assert far(got[0], y.detach()) < 0.01 and far(got[1], last.detach()) < 0.01
    for a, b, name in zip(got[2:], (grads[0], grads[1], grads[2], grads[3], grads[4], grads[5]), "x w b r i decay".split()):
        assert far(a, b) < 0.06, (name, far(a, b))


def test_two_streams_at_once(cf):
    a, b = block_inputs(21), block_inputs(22, rows=500, C=64)
    ra, rb = block(cf, a), block(cf, b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        qa, qb = block(cf, a, stream=s1), block(cf, b, stream=s2)
        assert all(t.is_cuda for t in qa)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(qa + qb, ra + rb))


def test_captured_and_replayed(cf):
    """Two graphs of the block, replayed in turn with other inputs, give what eager calls give."""
    a, b = block_inputs(31), block_inputs(32)
    block(cf, a)
    torch.cuda.synchronize()
    graphs = []
    for v in (a, b):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = block(cf, v)
        graphs.append((graph, v, out))
    for seed in (33, 34):
        for graph, v, out in graphs:
            new = block_inputs(seed)
            for k in v:
                v[k].copy_(new[k])
            graph.replay()
        torch.cuda.synchronize()
        for graph, v, out in graphs:
            assert all(torch.equal(p, q) for p, q in zip(out, block(cf, v)))


def test_steps_captured_and_replayed(cf):
    """A decoding step in a graph: the state moves on with each replay."""
    g = gen(41)
    B, C, T = 4, 128, 5
    xs, rs, is_ = (normal(g, B, T, C, dtype=torch.bfloat16).cuda() for _ in range(3))
    w, b = normal(g, C, 4, dtype=torch.bfloat16).cuda(), normal(g, C, dtype=torch.bfloat16).cuda()
    decay = torch.exp(torch.rand(C, generator=g) * 7 - 6).cuda()
    index = torch.tensor([5, 1, 0, 3], dtype=torch.int32).cuda()

    def step(window, h, x, r, i):
        return cf.gated_scan_step(cf.conv_causal_step(x, w, window, b, activation="silu", index=index), r, i, decay, h,
                                  index=index)

    window, h = torch.zeros(6, 3, C, dtype=torch.bfloat16).cuda(), torch.zeros(6, C).cuda()
    x, r, i = xs[:, 0].contiguous(), rs[:, 0].contiguous(), is_[:, 0].contiguous()
    step(window.clone(), h.clone(), x, r, i)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(window, h, x, r, i)
    window.zero_()
    h.zero_()
    ew, eh = window.clone(), h.clone()
    for t in range(T):
        for dst, src in ((x, xs), (r, rs), (i, is_)):
            dst.copy_(src[:, t])
        graph.replay()
        ref = step(ew, eh, xs[:, t], rs[:, t], is_[:, t])
        assert torch.equal(y, ref)
    assert torch.equal(window, ew) and torch.equal(h, eh)


def test_bad_offsets_stay_in_bounds(cf):
    """Offsets out of order or out of range: results unspecified, nothing outside the outputs written."""
    g = gen(51)
    rows, C = 200, 64
    x, r, i, dy = (normal(g, rows, C, dtype=torch.bfloat16).cuda() for _ in range(4))
    w, decay = normal(g, C, 4, dtype=torch.bfloat16).cuda(), torch.ones(C).cuda()
    state, h0 = normal(g, 4, 3, C, dtype=torch.bfloat16).cuda(), normal(g, 4, C, dtype=torch.float32).cuda()
    for cu in ([0, 150, 50, 120, 200], [-5, 10, 60, 300, 500], [30, 40, 50, 60, 70], [500, 600, 700, 800, 900],
               [0, -3, -3, 250, 100]):
        c = torch.tensor(cu, dtype=torch.int32).cuda()
        y, left = cf.conv_causal(x, w, state=state, cu_seqlens=c, return_state=True)
        cf.conv_causal_grad(x, w, dy, state=state, dstate_out=left, cu_seqlens=c, activation="silu")
        y, last, states = cf.gated_scan(x, r, i, decay, h0=h0, cu_seqlens=c, save_states=True)
        cf.gated_scan_grad(x, r, i, decay, dy, states, h0=h0, dh_last=h0, cu_seqlens=c)
        torch.cuda.synchronize()
    # rows in front of the first sequence are unused too
    c = torch.tensor([30, 40, 40, 90, 130], dtype=torch.int32).cuda()
    y, last, states = cf.gated_scan(x, r, i, decay, h0=h0, cu_seqlens=c, save_states=True)
    ref, rl = cf.gated_scan(x[30:], r[30:], i[30:], decay, h0=h0, cu_seqlens=c - 30)
    assert torch.allclose(y[30:].float(), ref.float(), atol=1e-2) and (y[:30] == 0).all() and torch.allclose(last, rl, atol=1e-5)
    z = cf.conv_causal(x, w, state=state, cu_seqlens=c)
    assert torch.equal(z[30:], cf.conv_causal(x[30:], w, state=state, cu_seqlens=c - 30)) and (z[:30] == 0).all()


def test_many_short_sequences(cf):
    """Batches past a grid dimension's 65535: as packed, and as their first and last sequences alone."""
    N, L, C = 70001, 2, 8
    torch.manual_seed(1)
    x, r, i, dy = (torch.randn(N, L, C, device="cuda").half() for _ in range(4))
    decay, w = torch.rand(C, device="cuda"), torch.randn(C, 4, device="cuda").half()
    ends = torch.tensor([0, 1, 65534, 65535, 65536, N - 1], device="cuda")
    y, last, states = cf.gated_scan(x, r, i, decay, save_states=True)
    part = [t[ends] for t in (x, r, i)]
    ys, ls, ss = cf.gated_scan(*part, decay, save_states=True)
    assert torch.equal(y[ends], ys) and torch.equal(last[ends], ls)
    grads, few = cf.gated_scan_grad(x, r, i, decay, dy, states), cf.gated_scan_grad(*part, decay, dy[ends], ss)
    assert all(torch.equal(a[ends], b) for a, b in zip(grads[:3], few[:3]))
    cu = (torch.arange(N + 1, device="cuda") * L).int()
    flat = [t.view(N * L, C) for t in (x, r, i, dy)]
    yp, lp, sp = cf.gated_scan(*flat[:3], decay, cu_seqlens=cu, save_states=True)
    assert torch.equal(yp, y.view(N * L, C)) and torch.equal(lp, last)
    gp = cf.gated_scan_grad(*flat[:3], decay, flat[3], sp, cu_seqlens=cu)
    assert all(torch.equal(a, b.view(N * L, C)) for a, b in zip(gp[:3], grads[:3]))
    z, left = cf.conv_causal(x, w, return_state=True)
    assert torch.equal(z[ends], cf.conv_causal(x[ends], w)) and torch.equal(left[:, 1:], x)
    assert torch.equal(cf.conv_causal(flat[0], w, cu_seqlens=cu), z.view(N * L, C))
    dx = cf.conv_causal_grad(x, w, dy)[0]
    assert torch.equal(dx[ends], cf.conv_causal_grad(x[ends], w, dy[ends])[0])
    # more runs of a convolution than one grid dimension holds
    big = (torch.randn(600_000, 1, C, device="cuda") / 16).half()
    z = cf.conv_causal(big, w)
    assert torch.equal(z[-5:], cf.conv_causal(big[-5:], w)) and torch.equal(z[530_000:530_005], cf.conv_causal(big[530_000:530_005], w))
    dx, dw, _, _ = cf.conv_causal_grad(big, w, big)
    assert torch.equal(dx[-5:], cf.conv_causal_grad(big[-5:], w, big[-5:])[0])
    ref = (big.double() ** 2).sum((0, 1))
    # squares: each of 75000 blocks' sums added in eight chains of 9375, and rounded to half: 9383 * 2^-24 + 2^-11
    assert torch.allclose(dw[:, 3].double(), ref, rtol=1.1e-3)


def test_offsets_past_31_bits(cf):
    """More than 2^31 elements: the far end of a long batch is computed as a short one is."""
    C, L = 65536, 33024
    torch.manual_seed(0)
    one = torch.randn(3, 1024, C, device="cuda").to(torch.bfloat16)
    x, r, i = (t.repeat(1 + L // 1024, 1)[None, :L] for t in one)
    decay = torch.full((C,), 0.7, device="cuda")
    y, last, states = cf.gated_scan(x, r, i, decay, save_states=True)
    assert y.numel() > 2 ** 31
    lo = (L - 1) // 64 * 64 - 64
    ref, rl = cf.gated_scan(x[:, lo:], r[:, lo:], i[:, lo:], decay, h0=states[:, lo // 64])
    assert torch.allclose(y[:, lo:].float(), ref.float(), rtol=2 ** -7, atol=1e-6) and torch.allclose(last, rl, rtol=1e-5, atol=1e-6)
    del y, ref, states, r, i
    w = torch.randn(C, 4, device="cuda").to(torch.bfloat16)
    z = cf.conv_causal(x, w)
    assert torch.equal(z[:, -60:], cf.conv_causal(x[:, -63:], w)[:, 3:])
    p = cf.act8_pack(x)
    q = cf.act8_pack(x[:, -5:])
    assert torch.equal(p.q[:, -5:], q.q) and torch.equal(p.scale[:, -5:], q.scale)

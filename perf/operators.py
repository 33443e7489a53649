"""The cases by which the sequence operators are measured, with their plain forms.

Operators: the causal depthwise convolution of a sequence (`conv_causal`, `conv_causal_grad`, `conv_causal_step`), the gated
linear recurrence (`gated_scan`, `gated_scan_grad`, `gated_scan_step`) and activation checkpoints in 8 bits (`act8_pack`,
`act8_unpack`), which the two gradients and `conv_wgrad` read in place of the 16-bit activations.

A batch is `n` sequences of `length` tokens, [n, length, C], or (where `packed`) `n` sequences of any lengths, some of them empty,
in [tokens, C], with the rows behind the last one unused: their outputs are zeros.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
STATE_EVERY = 64  # gated_scan_grad takes the recurrence's state in front of every 64th token


def listed():
    return [
        # one new token for each of 32 requests, their windows kept in a pool of slots: the smallest call of a serving loop
        dict(name="conv_step_32", op="conv_step", n=32, slots=48, C=2048, K=4, dtype="bf16", act=True),
        # the layer of an ordinary training batch or prompt
        dict(name="conv_4x2048", op="conv", n=4, length=2048, packed=False, C=2048, K=4, dtype="bf16", act=True, state=False),
        # prompts of any lengths packed end to end, a channel count that no vector divides, windows carried over from before
        dict(name="conv_packed_f32", op="conv", n=19, length=4099, packed=True, C=333, K=3, dtype="f32", act=False, state=True),
        # the gradient of a large training batch
        dict(name="conv_grad_8x4096", op="conv_grad", n=8, length=4096, packed=False, C=2560, K=4, dtype="bf16", act=True, state=False,
             saved8=False),
        # the same from 8-bit checkpoints, documents packed end to end, windows and their gradients carried
        dict(name="conv_grad_packed_8bit", op="conv_grad", n=37, length=12289, packed=True, C=1024, K=4, dtype="f16", act=True, state=True,
             saved8=True),
        # one new token for each of 128 requests
        dict(name="scan_step_128", op="scan_step", n=128, slots=160, C=4096, dtype="bf16"),
        # a short prompt in 32 bits: latency
        dict(name="scan_77_f32", op="scan", n=1, length=77, packed=False, C=256, dtype="f32", state=True, fused=False),
        # one long document, the gates two halves of one projection's output
        dict(name="scan_65536", op="scan", n=1, length=65536, packed=False, C=2048, dtype="bf16", state=False, fused=True),
        # the gradient of an ordinary training batch
        dict(name="scan_grad_4x4096", op="scan_grad", n=4, length=4096, packed=False, C=2560, dtype="bf16", state=False, saved8=False),
        # the same from 8-bit checkpoints, documents packed end to end
        dict(name="scan_grad_packed_8bit", op="scan_grad", n=29, length=16001, packed=True, C=2048, dtype="f16", state=True, saved8=True),
        # a large training batch's activations put into 8 bits and taken out again
        dict(name="act8_8x4096", op="act8", rows=32768, C=2560, dtype="bf16"),
        # the weight gradient of a 3x3 layer, 256 to 256 channels at 56 x 56, from its input's 8-bit checkpoint
        dict(name="wgrad_8bit", op="wgrad", n=64, H=56, W=56, C=256, O=256, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv_step", "conv", "conv_grad", "scan_step", "scan", "scan_grad", "act8", "wgrad"])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]))
    if op == "wgrad":  # layers that the tensor cores take
        c.update(dtype=rng.choice(["bf16", "f16"]), n=_log(rng, 1, 48), H=rng.randint(5, 56), W=rng.randint(5, 56), C=64 * rng.randint(1, 4), O=256)
        return c
    C = _log(rng, 32, 4096)
    c["C"] = C if rng.random() < 0.4 else max(16, C // 16 * 16)
    if op.endswith("_step"):
        c["n"] = _log(rng, 1, 512)
        c["slots"] = c["n"] + rng.randint(0, 64)
    elif op == "act8":
        c["rows"] = _log(rng, 1, max(2, min(40000, 60_000_000 // c["C"])))
    else:
        c["packed"] = rng.random() < 0.4
        tokens = _log(rng, 1, min(40000, 40_000_000 // c["C"]))
        c["n"] = _log(rng, 1, 40) if c["packed"] else min(tokens, _log(rng, 1, 16))
        c["length"] = tokens if c["packed"] else max(1, tokens // c["n"])
        c["state"] = rng.random() < 0.4
        if op.startswith("scan"):
            c["fused"] = rng.random() < 0.3
        if op.endswith("grad"):
            c["saved8"] = rng.random() < 0.4
    if op.startswith("conv"):
        c["K"] = rng.randint(2, 5)
        c["act"] = rng.random() < 0.6
    return c


# ---- inputs ------------------------------------------------------------------------------------------------------------------------


def _power_of_two(e):
    """2^e in 64 bits, by its bits: a library's exp2 need not be exact, and halves have to stay halves."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _pack8(v):
    """Whole numbers of up to 7 bits and their sign, and a power of two for each 32 channels (its exponent + 127): the least one by
    which the block's largest magnitude is at most 127."""
    top, C = torch.finfo(v.dtype).max, v.shape[-1]
    x = torch.nn.functional.pad(v.double(), (0, -C % 32)).unflatten(-1, (-1, 32))
    most, e = torch.frexp(x.abs().amax(-1) / 127)
    e = (e - (most == 0.5).to(e.dtype)).clamp(min=-126)
    e = torch.where(most == 0, torch.full_like(e, -127), e)
    step = _power_of_two(e).unsqueeze(-1)
    limit = torch.floor(top / step).clamp(max=127)
    q = torch.minimum(torch.maximum(torch.round(x / step), -limit), limit)
    return q.flatten(-2)[..., :C].to(torch.int8).contiguous(), (e + 127).to(torch.uint8)


def _unpack8(q, scale, dtype):
    step = (scale.to(torch.int32) << 23).view(torch.float32).to(dtype)  # the byte is a float's exponent
    return q.to(dtype) * step.repeat_interleave(32, -1)[..., : q.shape[-1]]


def _lengths(case, g):
    """Where each sequence begins, on the CPU: lengths of any size, empty ones and ones of a single token among them, and some rows
    behind the last."""
    n, T = case["n"], case["length"]
    if not case["packed"]:
        return torch.arange(n + 1) * T
    if n == 1:
        return torch.tensor([0, T - T // 50])
    cuts = torch.randint(0, T - T // 50 + 1, (n - 1,), generator=g).sort().values
    if n > 4:
        cuts[1] = cuts[0]
    if n > 6:
        cuts[4] = torch.minimum(cuts[3] + 1, cuts[5])
    return torch.cat([torch.tensor([0]), cuts, torch.tensor([T - T // 50])])


def prepare(case, seed):
    op, C, dt = case["op"], case["C"], DTYPES[case["dtype"]]
    host = torch.Generator().manual_seed(seed)
    g = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape, scale=1.0, shift=0.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * scale + shift).to(dtype)

    s = dict(case=case)
    if op == "act8":
        # activations as they come: a level of its own for each row, a few channels far above the others, rows of zeros
        s["x"] = normal(case["rows"], C)
        s["x"] *= torch.exp2(torch.randint(-6, 7, (case["rows"], 1), generator=g, device="cuda").float()).to(dt)
        s["x"] *= (torch.rand(C, generator=g, device="cuda") > 0.99).to(dt) * 15 + 1
        s["x"] *= (torch.rand(case["rows"], 1, generator=g, device="cuda") > 0.01).to(dt)
        return s
    if op == "wgrad":
        s["x8"] = _pack8(normal(case["n"], case["H"], case["W"], C))
        s["dy"] = normal(case["n"], case["H"], case["W"], case["O"])
        return s
    if op.startswith("conv"):
        s["w"] = normal(C, case["K"], scale=case["K"] ** -0.5)
        s["bias"] = normal(C, scale=0.3)
    else:
        # the gates of a trained layer: slow channels (a state that lives for a thousand tokens) and fast ones
        s["decay"] = torch.exp(torch.rand(C, generator=g, device="cuda") * math.log(8e3) + math.log(1e-3))
    if op.endswith("_step"):
        n, slots = case["n"], case["slots"]
        s["index"] = torch.randperm(slots, generator=host)[:n].to(torch.int32).cuda()
        s["x"] = normal(n, C)
        if op == "conv_step":
            s["pool"] = normal(slots, case["K"] - 1, C)
        else:
            s["r"], s["i"], s["pool"] = normal(n, C, scale=1.5), normal(n, C, scale=1.5, shift=0.5), normal(slots, C, dtype=torch.float32)
        return s

    n, packed = case["n"], case["packed"]
    cu = _lengths(case, host)
    s["cu"] = cu.to(torch.int32).cuda()
    tokens = case["length"] if packed else n * case["length"]
    # which sequence each token is in, its place there and that sequence's length (behind the last one: sequence n)
    at = torch.arange(tokens, device="cuda")
    edges = cu.cuda()
    s["seq"] = torch.searchsorted(edges[1:], at, right=True)
    s["used"] = s["seq"] < n
    own_seq = s["seq"].clamp(max=n - 1)
    s["pos"], s["len"] = at - edges[own_seq], (edges[1:] - edges[:-1])
    shape = (case["length"], C) if packed else (n, case["length"], C)
    inputs = dict(x=normal(*shape))
    if op.startswith("scan"):
        if case.get("fused"):
            gates = normal(*shape[:-1], 2 * C, scale=1.5)
            inputs["r"], inputs["i"] = gates[..., :C], gates[..., C:]
        else:
            inputs["r"], inputs["i"] = normal(*shape, scale=1.5), normal(*shape, scale=1.5, shift=0.5)
    saved8 = case.get("saved8", False)
    for k, v in inputs.items():
        s[k] = _pack8(v) if saved8 else v
    if case["state"]:
        s["h0"] = normal(n, C, dtype=torch.float32) if op.startswith("scan") else normal(n, case["K"] - 1, C)
    else:
        s["h0"] = None
    if op.endswith("grad"):
        s["dy"] = normal(*shape)
        s["dlast"] = (normal(n, C, dtype=torch.float32) if op.startswith("scan") else normal(n, case["K"] - 1, C)) if case["state"] else None
        if op == "scan_grad":
            # what the forward pass left: the state in front of every 64th token
            h = _scan_forward(s)[0].unflatten(0, (1, -1) if packed else (n, -1))
            before = torch.nn.functional.pad(h, (0, 0, 1, 0))[:, : h.shape[1]]
            s["states"] = before[:, ::STATE_EVERY].contiguous()
    return s


# ---- the plain forms ---------------------------------------------------------------------------------------------------------------


def _value(s, k, dtype=torch.float32):
    """An input as [tokens, C], out of its 8 bits where it is held in them."""
    v = s[k]
    v = _unpack8(*v, dtype) if isinstance(v, tuple) else v.to(dtype)
    return v.reshape(-1, v.shape[-1])


def _shifted(v, by):
    """v[t - by], zeros where there is none."""
    by = max(-v.shape[0], min(v.shape[0], by))
    zeros = v.new_zeros(abs(by), *v.shape[1:])
    return torch.cat([zeros, v[: v.shape[0] - by]]) if by >= 0 else torch.cat([v[-by:], zeros])


def _mask(keep, v):
    return torch.where(keep[:, None], v, torch.zeros_like(v))


def _tap(s, X, back):
    """x `back` tokens ago in the same sequence, or out of the window from before it."""
    K = s["case"]["K"]
    v = _mask(s["used"] & (s["pos"] >= back), _shifted(X, back))
    if s["h0"] is None or back == 0:
        return v
    old = s["h0"].float()[s["seq"].clamp(max=s["case"]["n"] - 1), (K - 1 + s["pos"] - back).clamp(0, K - 2)]
    return v + _mask(s["used"] & (s["pos"] < back), old)


def _before_activation(s, X):
    K, w = s["case"]["K"], s["w"].float()
    return s["bias"].float() + sum(w[:, j] * _tap(s, X, K - 1 - j) for j in range(K))


def _last_rows(s, X):
    """The window that each sequence leaves: its last K - 1 rows, older ones from the window before it."""
    K, n = s["case"]["K"], s["case"]["n"]
    j = torch.arange(K - 1, device=X.device)
    p = s["len"][:, None] + j - (K - 1)
    new = X[(s["cu"][:-1, None].long() + p).clamp(0, X.shape[0] - 1)]
    old = torch.zeros_like(new) if s["h0"] is None else s["h0"].float()[torch.arange(n, device=X.device)[:, None], (p + K - 1).clamp(max=K - 2)]
    return torch.where(p[..., None] >= 0, new, old)


def _conv_gradients(s):
    K, n, w = s["case"]["K"], s["case"]["n"], s["w"].float()
    X = _value(s, "x")
    dz = _value(s, "dy")
    if s["case"]["act"]:
        z = _before_activation(s, X)
        sig = torch.sigmoid(z)
        dz = dz * (sig * (1 + z * (1 - sig)))
    dz = _mask(s["used"], dz)
    length = s["len"][s["seq"].clamp(max=n - 1)]
    dx = sum(w[:, K - 1 - o] * _mask(s["used"] & (s["pos"] + o < length), _shifted(dz, -o)) for o in range(K))
    dw = torch.stack([(dz * _tap(s, X, K - 1 - j)).sum(0) for j in range(K)], 1)
    dbias, dstate = dz.sum(0), None
    if s["h0"] is not None:
        dlast, starts = s["dlast"].float(), s["cu"][:-1].long()
        slot = s["pos"] - length + K - 1
        dx = dx + _mask(s["used"] & (slot >= 0), dlast[s["seq"].clamp(max=n - 1), slot.clamp(0, K - 2)])
        m = torch.arange(K - 1, device=X.device)
        # old row m is read by the token at place p through the tap K - 1 + p - m tokens back
        dstate = sum((p < s["len"])[:, None, None] * (p <= m)[:, None] * w[:, (m - p).clamp(min=0)].T * dz[(starts + p).clamp(max=dz.shape[0] - 1)][:, None] for p in range(K - 1))
        j = m - s["len"][:, None]
        dstate = dstate + (j >= 0)[..., None] * dlast[torch.arange(n, device=X.device)[:, None], j.clamp(min=0)]
    return dx, dw, dbias, dstate


def _gates(s):
    X, sr, si = _value(s, "x"), torch.sigmoid(_value(s, "r")), torch.sigmoid(_value(s, "i"))
    log_a = -s["decay"] * sr
    # a next to 1 is raised to the power of thousands of tokens: it has to be rounded to nearest, which a library's exp need not do
    return X, sr, si, torch.exp(log_a.double()).float(), torch.sqrt(-torch.expm1(2 * log_a))


def _scan(a, u):
    """h[t] = a[t] h[t-1] + u[t] over dimension 0, by doubling."""
    by = 1
    while by < a.shape[0]:
        u = torch.cat([u[:by], u[by:] + a[by:] * u[:-by]])
        a = torch.cat([a[:by], a[by:] * a[:-by]])
        by *= 2
    return u


def _scan_forward(s):
    """The states [tokens, C] and what the gates were."""
    X, sr, si, a, m = _gates(s)
    first = (s["used"] & (s["pos"] == 0))[:, None]
    u = m * si * X
    if s["h0"] is not None:
        u = u + first * (a * s["h0"][s["seq"].clamp(max=s["case"]["n"] - 1)])
    h = _scan(torch.where(first | ~s["used"][:, None], torch.zeros_like(a), a), _mask(s["used"], u))
    return h, X, sr, si, a, m


def _scan_gradients(s):
    n = s["case"]["n"]
    h, X, sr, si, a, m = _scan_forward(s)
    at = s["seq"].clamp(max=n - 1)
    last = s["used"] & (s["pos"] == s["len"][at] - 1)
    dy = _mask(s["used"], _value(s, "dy"))
    if s["dlast"] is not None:
        dy = dy + _mask(last, s["dlast"][at])
    G = _scan(_mask(s["used"] & ~last, _shifted(a, -1)).flip(0), dy.flip(0)).flip(0)
    first = s["used"] & (s["pos"] == 0)
    before = _mask(~first, _shifted(h, 1))
    if s["h0"] is not None:
        before = before + _mask(first, s["h0"][at])
    dlog = a * G * (before - a * si * X / m)
    dx, di, dr = G * m * si, G * m * X * si * (1 - si), -s["decay"] * dlog * sr * (1 - sr)
    ddecay = -_mask(s["used"], sr * dlog).sum(0)
    dh0 = None
    if s["h0"] is not None:
        starts = s["cu"][:-1].long().clamp(max=a.shape[0] - 1)
        dh0 = torch.where((s["len"] > 0)[:, None], (a * G)[starts], s["dlast"])
    return tuple(_mask(s["used"], v) for v in (dx, dr, di)) + (ddecay, dh0)


def _outputs(names, values):
    return {k: v for k, v in zip(names, values) if v is not None}


def _plain(s):
    case = s["case"]
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op == "act8":
        q, scale = _pack8(s["x"])
        return dict(x=_unpack8(q, scale, torch.float32).to(dt), scale=scale)
    if op == "wgrad":
        n, H, W = case["n"], case["H"], case["W"]
        x = torch.nn.functional.pad(_unpack8(*s["x8"], torch.float32), (0, 0, 1, 1, 1, 1))
        dy = s["dy"].float().flatten(0, 2).T
        dw = [dy @ x[:, k // 3 : k // 3 + H, k % 3 : k % 3 + W].flatten(0, 2) for k in range(9)]
        return dict(dw=torch.stack(dw, 1).unflatten(1, (3, 3)).to(dt))
    if op == "conv_step":
        at = s["index"].long()
        rows = torch.cat([s["pool"][at], s["x"][:, None]], 1)
        z = s["bias"].float() + (rows.float() * s["w"].float().T).sum(1)
        s["pool"][at] = rows[:, 1:]
        return dict(y=(z * torch.sigmoid(z) if case["act"] else z).to(dt), pool=s["pool"])
    if op == "scan_step":
        at = s["index"].long()
        X, sr, si, a, m = _gates(s)
        h = a * s["pool"][at] + m * si * X
        s["pool"][at] = h
        return dict(y=h.to(dt), pool=s["pool"])
    shape = s["dy"].shape if op.endswith("grad") else s["x"].shape
    if op == "conv":
        X = _value(s, "x")
        z = _before_activation(s, X)
        y = _mask(s["used"], z * torch.sigmoid(z) if case["act"] else z).to(dt).view(shape)
        return _outputs(("y", "state"), (y, _last_rows(s, X).to(dt) if case["state"] else None))
    if op == "conv_grad":
        dx, dw, dbias, dstate = _conv_gradients(s)
        return _outputs(("dx", "dw", "dbias", "dstate"), (dx.to(dt).view(shape), dw.to(dt), dbias.to(dt), None if dstate is None else dstate.to(dt)))
    if op == "scan":
        h = _scan_forward(s)[0]
        ends = s["cu"][1:].long() - 1
        none = torch.zeros_like(h[:1]) if s["h0"] is None else s["h0"]
        last = torch.where((s["len"] > 0)[:, None], h[ends.clamp(min=0)], none)
        return dict(y=h.to(dt).view(shape), last=last)
    dx, dr, di, ddecay, dh0 = _scan_gradients(s)
    return _outputs(("dx", "dr", "di", "ddecay", "dh0"), tuple(v.to(dt).view(shape) for v in (dx, dr, di)) + (ddecay, dh0))


# ---- the framework's calls ---------------------------------------------------------------------------------------------------------


def _saved(s, k):
    import implicit_gemm_convolution_conv2d_b200 as cf

    return cf.Act8(*s[k], DTYPES[s["case"]["dtype"]]) if isinstance(s[k], tuple) else s[k]


def _framework(s):
    import implicit_gemm_convolution_conv2d_b200 as cf

    case = s["case"]
    op = case["op"]
    if op == "act8":
        p = cf.act8_pack(s["x"])
        return dict(x=cf.act8_unpack(p), scale=p.scale)
    if op == "wgrad":
        return dict(dw=cf.conv_wgrad(cf.Act8(*s["x8"], s["dy"].dtype), s["dy"], 3, padding=1))
    if op == "scan_step":
        return dict(y=cf.gated_scan_step(s["x"], s["r"], s["i"], s["decay"], s["pool"], index=s["index"]), pool=s["pool"])
    cu = s["cu"] if case.get("packed") else None
    if op.startswith("scan"):
        if op == "scan":
            y, last, _ = cf.gated_scan(s["x"], s["r"], s["i"], s["decay"], h0=s["h0"], cu_seqlens=cu, save_states=True)
            return dict(y=y, last=last)
        got = cf.gated_scan_grad(_saved(s, "x"), _saved(s, "r"), _saved(s, "i"), s["decay"], s["dy"], s["states"], h0=s["h0"],
                                 dh_last=s["dlast"], cu_seqlens=cu)
        return _outputs(("dx", "dr", "di", "ddecay", "dh0"), got)
    act = "silu" if case["act"] else None
    if op == "conv_step":
        return dict(y=cf.conv_causal_step(s["x"], s["w"], s["pool"], s["bias"], activation=act, index=s["index"]), pool=s["pool"])
    if op == "conv":
        if case["state"]:
            y, state = cf.conv_causal(s["x"], s["w"], s["bias"], activation=act, state=s["h0"], cu_seqlens=cu, return_state=True)
            return dict(y=y, state=state)
        return dict(y=cf.conv_causal(s["x"], s["w"], s["bias"], activation=act, cu_seqlens=cu))
    got = cf.conv_causal_grad(_saved(s, "x"), s["w"], s["dy"], s["bias"], activation=act, state=s["h0"], dstate_out=s["dlast"], cu_seqlens=cu)
    return _outputs(("dx", "dw", "dbias", "dstate"), got)


def run(state):
    return _framework(state) if own else _plain(state)


# ---- what a pass cannot do without -------------------------------------------------------------------------------------------------


def work(case):
    op, C, e = case["op"], case["C"], 4 if case["dtype"] == "f32" else 2
    eight = 1 + 1 / 32
    if op == "act8":
        return dict(bytes=case["rows"] * C * (2 * e + eight), flops=case["rows"] * C * 4)
    if op == "wgrad":
        pixels = case["n"] * case["H"] * case["W"]
        return dict(bytes=pixels * (C * eight + case["O"] * e) + 9 * C * case["O"] * e, flops=2 * 9 * pixels * C * case["O"])
    if op == "conv_step":
        return dict(bytes=case["n"] * C * e * (2 + 2 * (case["K"] - 1)) + C * e * (case["K"] + 1), flops=case["n"] * C * 2 * case["K"])
    if op == "scan_step":
        return dict(bytes=case["n"] * C * (4 * e + 8) + 4 * C, flops=case["n"] * C * 16)
    size = case["length"] * C * (1 if case["packed"] else case["n"])
    saved = eight if case.get("saved8") else e
    once = {"conv": 2 * e, "conv_grad": saved + 2 * e, "scan": 4 * e, "scan_grad": 3 * saved + 4 * e}[op]
    flops = {"conv": 2 * case.get("K", 0) + 4, "conv_grad": 6 * case.get("K", 0) + 8, "scan": 16, "scan_grad": 40}[op]
    row = case["n"] * C
    small = {"conv": row * (case.get("K", 1) - 1) * e * 2, "conv_grad": row * (case.get("K", 1) - 1) * e * 3, "scan": row * 8, "scan_grad": row * 12}[op]
    return dict(bytes=size * once + (small if case["state"] else 0), flops=size * flops)


# ---- the definitions in 64 bits ----------------------------------------------------------------------------------------------------


def exact(case, seed):
    """Token by token, each sequence by itself, as the formulas say it."""
    s = prepare(case, seed)
    op, C = case["op"], case["C"]
    f64 = lambda v: v.double()  # noqa: E731
    powers = torch.tensor([math.ldexp(1.0, k - 127) for k in range(256)], dtype=torch.float64, device="cuda")

    def whole(v):
        if not isinstance(v, tuple):
            return v.double()
        q, scale = v
        return q.double() * powers[scale.long()].repeat_interleave(32, -1)[..., : q.shape[-1]]

    if op == "act8":
        x, out, scales = s["x"].double(), [], []
        top = torch.finfo(s["x"].dtype).max
        for c in range(0, C, 32):
            b = x[:, c : c + 32]
            most = b.abs().max(1, keepdim=True).values
            e = torch.full_like(most, -126)
            for k in range(-126, 122):  # the least exponent that holds the block
                e = torch.where(most > 127 * 2.0**k, torch.full_like(e, k + 1), e)
            step = powers[(e + 127).long()]
            out.append(torch.minimum(torch.maximum(torch.round(b / step), -torch.floor(top / step)), torch.floor(top / step)).clamp(-127, 127) * step)
            scales.append(torch.where(most == 0, torch.zeros_like(e), e + 127))
        return dict(x=torch.cat(out, 1), scale=torch.cat(scales, 1).to(torch.uint8))
    if op == "wgrad":
        n, H, W, dw = case["n"], case["H"], case["W"], torch.zeros(case["O"], 3, 3, C, dtype=torch.float64, device="cuda")
        x, dy = whole(s["x8"]), f64(s["dy"])
        for kh in range(3):
            for kw in range(3):
                h0, h1, w0, w1 = max(0, 1 - kh), min(H, H + 1 - kh), max(0, 1 - kw), min(W, W + 1 - kw)
                a = dy[:, h0:h1, w0:w1].reshape(-1, case["O"])
                dw[:, kh, kw] = a.T @ x[:, h0 + kh - 1 : h1 + kh - 1, w0 + kw - 1 : w1 + kw - 1].reshape(-1, C)
        return dict(dw=dw)
    silu = lambda z: z / (1 + torch.exp(-z))  # noqa: E731
    if op == "conv_step":
        pool, at = f64(s["pool"]).clone(), s["index"].long()
        window = torch.cat([pool[at], f64(s["x"])[:, None]], 1)
        z = f64(s["bias"]) + torch.einsum("nkc,ck->nc", window, f64(s["w"]))
        pool[at] = window[:, 1:]
        return dict(y=silu(z) if case["act"] else z, pool=pool)
    if op == "scan_step":
        pool, at = f64(s["pool"]).clone(), s["index"].long()
        la = -f64(s["decay"]) / (1 + torch.exp(-f64(s["r"])))
        pool[at] = torch.exp(la) * pool[at] + torch.sqrt(-torch.expm1(2 * la)) / (1 + torch.exp(-f64(s["i"]))) * f64(s["x"])
        return dict(y=pool[at], pool=pool)

    n = case["n"]
    edges = s["cu"].tolist()
    x = whole(s["x"])
    rows = [(x[k],) if not case["packed"] else (x[edges[k] : edges[k + 1]],) for k in range(n)]
    part = (lambda v, k: v[k]) if not case["packed"] else (lambda v, k: v[edges[k] : edges[k + 1]])

    def joined(parts):
        if not case["packed"]:
            return torch.stack(parts)
        v = torch.cat(parts)
        return torch.cat([v, v.new_zeros(case["length"] - v.shape[0], C)])

    if op.startswith("conv"):
        K, w, b = case["K"], f64(s["w"]), f64(s["bias"])
        ys, states, dxs, dws, dbs, dstates = [], [], [], [], [], []
        for k in range(n):
            L = rows[k][0].shape[0]
            old = f64(s["h0"][k]) if s["h0"] is not None else x.new_zeros(K - 1, C)
            ext = torch.cat([old, rows[k][0]])
            z = b + sum(ext[j : j + L] * w[:, j] for j in range(K))
            if op == "conv":
                ys.append(silu(z) if case["act"] else z)
                states.append(ext[L:])
                continue
            dz = part(f64(s["dy"]), k)
            if case["act"]:
                sg = 1 / (1 + torch.exp(-z))
                dz = dz * (sg + z * sg * (1 - sg))
            dext = torch.zeros_like(ext)
            for j in range(K):
                dext[j : j + L] += dz * w[:, j]
            if s["dlast"] is not None:
                dext[L:] += f64(s["dlast"][k])
            dxs.append(dext[K - 1 :])
            dstates.append(dext[: K - 1])
            dws.append(torch.stack([(dz * ext[j : j + L]).sum(0) for j in range(K)], 1))
            dbs.append(dz.sum(0))
        if op == "conv":
            return _outputs(("y", "state"), (joined(ys), torch.stack(states) if case["state"] else None))
        return _outputs(("dx", "dw", "dbias", "dstate"), (joined(dxs), sum(dws), sum(dbs), torch.stack(dstates) if case["state"] else None))

    # the recurrence, one token after the other, all sequences of a batch (or the whole packed row of them) at once
    first = set(edges[:-1]) if case["packed"] else {0}
    flat = (lambda v: v[None]) if case["packed"] else (lambda v: v)
    x, r, i = (flat(whole(s[k])) for k in ("x", "r", "i"))
    B, T = x.shape[:2]
    sr, si = 1 / (1 + torch.exp(-r)), 1 / (1 + torch.exp(-i))
    la = -f64(s["decay"]) * sr
    a, m = torch.exp(la), torch.sqrt(-torch.expm1(2 * la))
    u, stop = m * si * x, edges[-1] if case["packed"] else T
    seq = s["seq"].tolist() if case["packed"] else None
    zero = x.new_zeros(B, C)
    begin = lambda t: zero if s["h0"] is None else f64(s["h0"][seq[t]])[None] if case["packed"] else f64(s["h0"])  # noqa: E731
    h, before, now = torch.zeros_like(x), torch.zeros_like(x), zero
    for t in range(stop):
        if t in first:
            now = begin(t)
        before[:, t] = now
        now = torch.addcmul(u[:, t], a[:, t], now)
        h[:, t] = now
    back = (lambda v: v[0]) if case["packed"] else (lambda v: v)
    if op == "scan":
        if not case["packed"]:
            last = h[:, -1]
        else:
            rest = torch.zeros(n, C, dtype=torch.float64, device="cuda") if s["h0"] is None else f64(s["h0"])
            last = torch.stack([h[0, edges[k + 1] - 1] if edges[k + 1] > edges[k] else rest[k] for k in range(n)])
        return dict(y=back(h), last=last)
    G, dy, carry = torch.zeros_like(x), flat(f64(s["dy"])), zero
    ends = {edges[k + 1] - 1: k for k in range(n) if edges[k + 1] > edges[k]} if case["packed"] else {T - 1: None}
    dh0 = f64(s["dlast"]).clone() if s["dlast"] is not None else None
    for t in range(stop - 1, -1, -1):
        if t in ends:
            carry = zero if s["dlast"] is None else f64(s["dlast"]) if ends[t] is None else f64(s["dlast"][ends[t]])[None]
        now = dy[:, t] + carry
        G[:, t] = now
        carry = a[:, t] * now
        if dh0 is not None and t in first:
            if case["packed"]:
                dh0[seq[t]] = carry[0]
            else:
                dh0 = carry
    dla = G * (a * before - a * a / m * si * x)
    dla[:, stop:] = 0
    dr, di = -f64(s["decay"]) * dla * sr * (1 - sr), G * m * x * si * (1 - si)
    return _outputs(("dx", "dr", "di", "ddecay", "dh0"), (back(G * m * si), back(dr), back(di), -(sr * dla).sum((0, 1)), dh0))

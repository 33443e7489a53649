"""Plain 64-bit forms of the sequence operators, token by token, with bounds of
what an fp32 kernel may be off by.

Gradients come from torch's double-precision autograd of the forward forms, so
they share no formula with the kernels.  Bounds count rounding units u = 2^-24:
sums and products one each; the fast exponential and division of CUDA's
programming guide, __expf(v) 2 + 1.173 |v| ulp and __fdividef 2 ulp (an ulp is
two units).  A result rounded to a 16-bit type is off by half a step more.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def smallest(dtype):
    """Half of the spacing at zero: what a subnormal result may be off by."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def worst(got, ref, bound, dtype):
    """The largest |got - ref| over its bound (a rounding to `dtype` more); above 1 is a failure."""
    got, ref, bound = got.detach().cpu().double(), ref.detach(), bound.detach()
    assert got.shape == ref.shape, (got.shape, ref.shape)
    if got.numel() == 0:
        return 0.0
    assert torch.equal(torch.isfinite(got), torch.isfinite(ref)), "finite where the reference is not, or the reverse"
    fine = torch.isfinite(ref)
    limit = half_step(dtype) * (ref.abs() + bound) + bound + smallest(dtype)
    off = torch.where(fine, (got - ref).abs() / limit, torch.zeros_like(ref))
    return float(off.max())


# ---- sequences ----------------------------------------------------------


def ranges(N, L, cu):
    """(batch entry, first, behind the last) of each sequence."""
    if cu is None:
        return [(n, 0, L) for n in range(N)]
    return [(0, int(cu[k]), int(cu[k + 1])) for k in range(len(cu) - 1)]


def as_batch(t, cu):
    """[N, L, C] of a batch, [1, rows, C] of a packed run."""
    return t if cu is None else t[None]


# ---- 8-bit checkpoints --------------------------------------------------


POWERS = torch.tensor([2.0 ** (k - 127) for k in range(256)], dtype=torch.float64)  # by a step's byte


def act8(x):
    """(q, scale bytes) by the definition, in 64 bits and exact powers of two."""
    top, C = torch.finfo(x.dtype).max, x.shape[-1]
    v = torch.nn.functional.pad(x.double(), (0, -C % 32)).unflatten(-1, (-1, 32))
    amax = v.abs().amax(-1)
    bad = ~torch.isfinite(v).all(-1)
    amax = torch.where(bad, torch.zeros_like(amax), amax)
    man, e = torch.frexp(amax / 127)
    e = torch.where(man == 0.5, e - 1, e).clamp(min=-126)
    step = POWERS[e + 127].unsqueeze(-1)
    limit = torch.floor(top / step).clamp(max=127)
    q = torch.minimum(torch.maximum(torch.round(v / step), -limit), limit)
    q = torch.where(bad.unsqueeze(-1), torch.zeros_like(q), q)
    byte = torch.where(bad, torch.full_like(e, 255), torch.where(amax == 0, torch.zeros_like(e), e + 127))
    return q.flatten(-2)[..., :C].to(torch.int8), byte.to(torch.uint8)


def act8_values(q, scale):
    """The 64-bit values that a checkpoint stands for."""
    byte = scale.long()
    step = torch.where(byte == 255, torch.full((), float("nan"), dtype=torch.float64), POWERS[byte])
    return q.double() * step.repeat_interleave(32, -1)[..., : q.shape[-1]]


# ---- causal convolution -------------------------------------------------


def conv_causal(x, w, bias, silu, state, cu):
    """y (zeros in unused rows), the windows left behind, z and sum |w x| (64 bits in, 64 bits out)."""
    X, K, C = as_batch(x, cu), w.shape[1], w.shape[0]
    N, L = (x.shape[0], x.shape[1]) if cu is None else (len(cu) - 1, x.shape[0])
    zs = [torch.zeros_like(r) for r in X]
    S = [torch.zeros_like(r) for r in X]
    pieces, left = [[] for _ in X], []
    at = [0] * len(X)
    for k, (n, lo, hi) in enumerate(ranges(N, L, cu)):
        old = state[k] if state is not None else x.new_zeros(K - 1, C)
        ext = torch.cat([old, X[n][lo:hi]])
        T = hi - lo
        b = bias if bias is not None else x.new_zeros(C)
        z = b + sum(w[:, j] * ext[j : j + T] for j in range(K))
        s = b.abs() + sum((w[:, j] * ext[j : j + T]).abs() for j in range(K))
        pieces[n] += [x.new_zeros(lo - at[n], C), z]
        S[n][lo:hi] = s.detach()
        zs[n][lo:hi] = z.detach()
        at[n] = hi
        left.append(ext[T:])
    z = torch.stack([torch.cat(p + [x.new_zeros(L - at[n], C)]) for n, p in enumerate(pieces)])
    used = torch.zeros(z.shape[:2], dtype=torch.bool)
    for n, lo, hi in ranges(N, L, cu):
        used[n, lo:hi] = True
    y = torch.where(used[..., None], z * torch.sigmoid(z) if silu else z, torch.zeros_like(z))
    out = torch.stack(left) if left else x.new_zeros(0, K - 1, C)
    pick = (lambda t: t) if cu is None else (lambda t: t[0])
    return pick(y), out, pick(torch.stack(zs)) if zs else x * 0, pick(torch.stack(S)) if S else x * 0


def sigmoid_units(v):
    """Relative error of the kernels' sigmoid, in units: the exponential's where it is not small beside 1, the sum, the division."""
    return 2 * (2 + 1.173 * v.abs()) * torch.sigmoid(-v) + 6


def conv_bound(z, S, K, silu):
    b = U * (K + 2) * S
    if silu:  # |d silu| <= 1.1; the sigmoid and the product
        b = 1.1 * b + U * (sigmoid_units(z) + 2) * (z * torch.sigmoid(z)).abs()
    return b


def slope_bound(z, S, K):
    """Absolute error of d silu / dz = s (1 + z (1 - s)), whose own slope is at most 1/2."""
    s = torch.sigmoid(z)
    ks = sigmoid_units(z)
    return 0.5 * U * (K + 2) * S + U * ((ks + 4) * s * (1 + z.abs() * (1 - s)) + s * z.abs() * (s * ks + 2))


# ---- gated recurrence ---------------------------------------------------


def gates(r, i, decay):
    s, g = torch.sigmoid(r), torch.sigmoid(i)
    l = -decay * s
    return s, g, l, torch.exp(l), torch.sqrt(-torch.expm1(2 * l))


def gated_scan(x, r, i, decay, h0, cu):
    """y (zeros in unused rows), last states, states in front of every 64th token."""
    X, R, I = (as_batch(t, cu) for t in (x, r, i))
    N, L, C = (len(cu) - 1 if cu is not None else x.shape[0]), X.shape[1], X.shape[2]
    s, g, l, a, m = gates(R, I, decay)
    u = m * g * X
    rows = [[x.new_zeros(C)] * L for _ in range(X.shape[0])]
    last = []
    for k, (n, lo, hi) in enumerate(ranges(N, L, cu)):
        h = h0[k] if h0 is not None else x.new_zeros(C)
        for t in range(lo, hi):
            h = a[n, t] * h + u[n, t]
            rows[n][t] = h
        last.append(h)
    y = torch.stack([torch.stack(p) if p else x.new_zeros(0, C) for p in rows]) if rows else X * 0
    last = torch.stack(last) if last else x.new_zeros(0, C)
    return (y if cu is None else y[0]), last


def states_of(y, cu):
    """What save_states leaves where it has a meaning: the state in front of rows 64, 128, ... (0 in front of the first)."""
    Y = as_batch(y, cu).detach()
    return torch.nn.functional.pad(Y, (0, 0, 1, 0))[:, : Y.shape[1]][:, ::64]


def scan_units(r, i, decay):
    """Relative units of s, g, a, m and of u = m g x."""
    s, g, l, a, m = gates(r, i, decay)
    ks, kg = sigmoid_units(r), sigmoid_units(i)
    near = l > -0.25
    ka = l.abs() * (ks + 1) + 2 + torch.where(near, torch.zeros_like(l), 2 * (2 + 1.173 * l.abs()))
    # 1 - a: the series' own steps where a is next to 1, the rounding of a over 1 - a elsewhere; then 1 - a^2 and its root
    kE = ks + 1 + torch.where(near, torch.full_like(l, 6.0), ka * a / (1 - a))
    km = (kE + 4) / 2 + 2
    return ks, kg, ka, km, km + kg + 2


def scan_bounds(x, r, i, decay, h0, cu, dy=None, dh_last=None):
    """Bounds of h, and with dy of the gradients, by running the recurrences on magnitudes."""
    X, R, I = (as_batch(t, cu) for t in (x, r, i))
    N, L, C = (len(cu) - 1 if cu is not None else x.shape[0]), X.shape[1], X.shape[2]
    s, g, l, a, m = gates(R, I, decay)
    ks, kg, ka, km, ku = scan_units(R, I, decay)
    u = (m * g * X).abs()
    H, B = torch.zeros_like(X), torch.zeros_like(X)  # sum of magnitudes, and what h is off by
    Hp, Bp = torch.zeros_like(X), torch.zeros_like(X)
    zero = x.new_zeros(C)
    lastB = []
    for k, (n, lo, hi) in enumerate(ranges(N, L, cu)):
        h, b = (h0[k].abs() if h0 is not None else zero), zero
        for t in range(lo, hi):
            Hp[n, t], Bp[n, t] = h, b
            # the kernel may take a segment's product of a's and its own sum apart: two roundings more a step
            b = a[n, t] * b + U * ((ka[n, t] + 4) * a[n, t] * h + (ku[n, t] + 4) * u[n, t])
            h = a[n, t] * h + u[n, t]
            H[n, t], B[n, t] = h, b
        lastB.append(b)
    pick = (lambda t: t) if cu is None else (lambda t: t[0])
    res = {"y": pick(B), "last": torch.stack(lastB) if lastB else x.new_zeros(0, C)}
    if dy is None:
        return res
    D = as_batch(dy, cu).abs()
    G, BG = torch.zeros_like(X), torch.zeros_like(X)
    dh0 = []
    for k, (n, lo, hi) in enumerate(ranges(N, L, cu)):
        c, b = (dh_last[k].abs() if dh_last is not None else zero), zero
        for t in range(hi - 1, lo - 1, -1):
            G[n, t] = D[n, t] + c
            BG[n, t] = b + 2 * U * G[n, t]
            c = a[n, t] * G[n, t]
            b = a[n, t] * BG[n, t] + U * (ka[n, t] + 4) * c
        dh0.append(b)
    v = g * X.abs()
    res["dx"] = pick(m * g * BG + U * (km + kg + 3) * G * m * g)
    k1 = (1 - g) * m * v
    res["di"] = pick(k1 * BG + U * G * m * v * ((km + kg + 5) * (1 - g) + g * (kg + 2)))
    back = torch.where(m > 0, a * v / m, torch.zeros_like(m))
    inner = Hp + back
    dl = a * (BG * inner + G * (Bp + U * (ka + kg + km + 6) * back) + U * (ka + 4) * G * inner)
    mag = a * G * inner
    res["dr"] = pick(decay * s * ((1 - s) * dl + U * mag * ((ks + 5) * (1 - s) + s * (ks + 2))))
    # a sum of n terms in chains of at most 512 additions
    res["ddecay"] = (s * (dl + U * (ks + 2 + 512) * mag)).sum((0, 1))
    res["dh0"] = torch.stack(dh0) if dh0 else x.new_zeros(0, C)
    return res

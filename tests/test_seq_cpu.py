"""The sequence operators' host side and their 64-bit reference, without a GPU."""
from __future__ import annotations

import ctypes
import os
import re
import subprocess

import pytest
import torch

import tests.seq_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, EINVAL, EDTYPE, EALIGN, EALIAS = 0, -1, -2, -3, -4
BF16 = 2
P = 1 << 20  # addresses that no check refuses; nothing is queued where one does


@pytest.fixture(scope="module")
def L():
    from implicit_gemm_convolution_conv2d_b200 import _build, seq
    _build.build()
    return seq._lib()


def at(k):
    return P * (k + 1) * 64


def test_library_exports_every_declared_symbol(L):
    import implicit_gemm_convolution_conv2d_b200 as cf
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "conv_seq.h")).read(), flags=re.S)
    names = set(re.findall(r"^int\s+(\w+)\s*\(", text, flags=re.M))
    assert names == set(L) and len(names) == 10
    nm = subprocess.run(["nm", "-D", "--defined-only", cf.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert names <= {ln.split()[-1] for ln in nm.splitlines() if ln.strip()}


def test_header_compiles_as_c():
    src = "#include \"conv_seq.h\"\nint main(void) { return GATED_SCAN_STATE_EVERY + ACT8_BLOCK + CONV_ACT_SILU; }\n"
    r = subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-x", "c", "-", "-fsyntax-only"],
                       input=src, text=True, capture_output=True)
    assert r.returncode == 0, r.stderr


# argument lists that pass every check up to the launch, by name
def conv_args(**k):
    a = dict(x=at(0), w=at(1), bias=at(2), state=at(3), cu=None, y=at(4), state_out=at(5), N=2, L=10, C=16, K=4, xb=160, xt=16,
             act=1, fill=1, dtype=BF16, stream=None)
    a.update(k)
    return list(a.values())


def conv_grad_args(**k):
    a = dict(x=at(0), xs=None, w=at(1), bias=at(2), state=at(3), cu=None, dy=at(4), dso=at(5), dx=at(6), dw=at(7), db=at(8), ds=at(9),
             N=2, L=10, C=16, K=4, xb=160, xt=16, yb=160, yt=16, act=1, fill=1, dtype=BF16, ws=at(10), wb=1 << 20, stream=None)
    a.update(k)
    return list(a.values())


def conv_step_args(**k):
    a = dict(x=at(0), w=at(1), bias=at(2), state=at(3), index=at(4), y=at(5), B=3, slots=8, C=16, K=4, xt=16, act=1, fill=1,
             dtype=BF16, stream=None)
    a.update(k)
    return list(a.values())


def scan_args(**k):
    a = dict(x=at(0), r=at(1), i=at(2), decay=at(3), h0=at(4), cu=None, y=at(5), last=at(6), states=at(7), N=2, L=10, C=16, xb=160,
             xt=16, rb=160, rt=16, ib=160, it=16, fill=1, dtype=BF16, stream=None)
    a.update(k)
    return list(a.values())


def scan_grad_args(**k):
    a = dict(x=at(0), xs=None, r=at(1), rs=None, i=at(2), is_=None, decay=at(3), states=at(4), h0=at(5), cu=None, dy=at(6),
             dhl=at(7), dx=at(8), dr=at(9), di=at(10), dd=at(11), dh0=at(12), N=2, L=10, C=16, xb=160, xt=16, rb=160, rt=16,
             ib=160, it=16, yb=160, yt=16, fill=1, dtype=BF16, ws=at(13), wb=1 << 20, stream=None)
    a.update(k)
    return list(a.values())


def scan_step_args(**k):
    a = dict(x=at(0), r=at(1), i=at(2), decay=at(3), h=at(4), index=at(5), y=at(6), B=3, slots=8, C=16, xt=16, rt=16, it=16, fill=1,
             dtype=BF16, stream=None)
    a.update(k)
    return list(a.values())


def pack_args(**k):
    a = dict(x=at(0), q=at(1), scale=at(2), rows=5, C=40, xr=40, dtype=BF16, stream=None)
    a.update(k)
    return list(a.values())


def unpack_args(**k):
    a = dict(q=at(0), scale=at(1), y=at(2), rows=5, C=40, dtype=BF16, stream=None)
    a.update(k)
    return list(a.values())


REFUSED = [
    ("conv_causal", conv_args, [
        (dict(dtype=9), EDTYPE), (dict(K=0), EINVAL), (dict(K=9), EINVAL), (dict(C=0), EINVAL), (dict(N=-1), EINVAL),
        (dict(L=-1), EINVAL), (dict(L=1 << 31), EINVAL), (dict(L=(1 << 31) - 4096), EINVAL), (dict(act=2), EINVAL), (dict(x=None), EINVAL), (dict(w=None), EINVAL),
        (dict(y=None), EINVAL), (dict(xt=-1), EINVAL), (dict(xb=-1), EINVAL), (dict(xt=1 << 60), EINVAL), (dict(x=at(0) + 1), EALIGN),
        (dict(y=at(4) + 1), EALIGN), (dict(cu=at(6) + 2), EALIGN), (dict(y=at(0) + 64), EALIAS), (dict(state_out=at(3)), EALIAS),
        (dict(y=at(1)), EALIAS), (dict(state_out=at(4) + 32), EALIAS)]),
    ("conv_causal_grad", conv_grad_args, [
        (dict(dtype=-1), EDTYPE), (dict(K=9), EINVAL), (dict(ws=None), EINVAL), (dict(wb=16), EINVAL), (dict(dw=None), EINVAL),
        (dict(db=None), EINVAL), (dict(dx=None), EINVAL), (dict(dy=None), EINVAL), (dict(state=None), EINVAL), (dict(act=-1), EINVAL),
        (dict(ws=at(10) + 4), EALIGN), (dict(dy=at(4) + 1), EALIGN), (dict(dx=at(4)), EALIAS), (dict(dx=at(0)), EALIAS),
        (dict(dw=at(1)), EALIAS), (dict(ds=at(5)), EALIAS), (dict(ws=at(6)), EALIAS), (dict(yt=-16), EINVAL)]),
    ("conv_causal_step", conv_step_args, [
        (dict(dtype=3), EDTYPE), (dict(B=-1), EINVAL), (dict(slots=-1), EINVAL), (dict(K=9), EINVAL), (dict(index=None, slots=2), EINVAL),
        (dict(state=None), EINVAL), (dict(y=None), EINVAL), (dict(act=7), EINVAL), (dict(index=at(4) + 1), EALIGN),
        (dict(state=at(3) + 1), EALIGN), (dict(y=at(0)), EALIAS), (dict(y=at(3)), EALIAS), (dict(state=at(1)), EALIAS)]),
    ("gated_scan", scan_args, [
        (dict(dtype=4), EDTYPE), (dict(C=-4), EINVAL), (dict(N=-2), EINVAL), (dict(L=1 << 31), EINVAL), (dict(decay=None), EINVAL),
        (dict(y=None), EINVAL), (dict(r=None), EINVAL), (dict(it=-1), EINVAL), (dict(i=at(2) + 1), EALIGN), (dict(states=at(7) + 2), EALIGN),
        (dict(decay=at(3) + 1), EALIGN), (dict(y=at(0)), EALIAS), (dict(y=at(1) + 320), EALIAS), (dict(last=at(4)), EALIAS),
        (dict(states=at(5)), EALIAS), (dict(N=1 << 30, L=1 << 30, C=1 << 20), EINVAL)]),
    ("gated_scan_grad", scan_grad_args, [
        (dict(dtype=4), EDTYPE), (dict(states=None), EINVAL), (dict(dd=None), EINVAL), (dict(dr=None), EINVAL), (dict(ws=None), EINVAL),
        (dict(wb=8), EINVAL), (dict(x=None), EINVAL), (dict(yt=-1), EINVAL), (dict(dh0=at(12) + 2), EALIGN), (dict(dx=at(8) + 1), EALIGN),
        (dict(dx=at(0)), EALIAS), (dict(dr=at(8)), EALIAS), (dict(di=at(6)), EALIAS), (dict(dh0=at(7)), EALIAS), (dict(ws=at(4)), EALIAS),
        (dict(dd=at(3)), EALIAS)]),
    ("gated_scan_step", scan_step_args, [
        (dict(dtype=3), EDTYPE), (dict(B=-1), EINVAL), (dict(index=None, slots=1), EINVAL), (dict(h=None), EINVAL), (dict(decay=None), EINVAL),
        (dict(y=None), EINVAL), (dict(h=at(4) + 1), EALIGN), (dict(y=at(0)), EALIAS), (dict(h=at(3)), EALIAS), (dict(y=at(4)), EALIAS)]),
    ("act8_pack", pack_args, [
        (dict(dtype=3), EDTYPE), (dict(rows=-1), EINVAL), (dict(C=0), EINVAL), (dict(xr=-1), EINVAL), (dict(x=None), EINVAL),
        (dict(q=None), EINVAL), (dict(scale=None), EINVAL), (dict(x=at(0) + 1), EALIGN), (dict(q=at(0)), EALIAS), (dict(scale=at(1) + 8), EALIAS)]),
    ("act8_unpack", unpack_args, [
        (dict(dtype=3), EDTYPE), (dict(rows=-1), EINVAL), (dict(C=0), EINVAL), (dict(y=None), EINVAL), (dict(y=at(2) + 1), EALIGN),
        (dict(y=at(0)), EALIAS), (dict(y=at(1)), EALIAS)]),
]


@pytest.mark.parametrize("name,args,cases", REFUSED, ids=[r[0] for r in REFUSED])
def test_refusals(L, name, args, cases):
    for change, code in cases:
        assert L[name](*args(**change)) == code, (name, change)


def test_nothing_to_do(L):
    assert L["conv_causal"](*conv_args(N=0)) == OK
    assert L["conv_causal_step"](*conv_step_args(B=0)) == OK
    assert L["gated_scan"](*scan_args(N=0)) == OK
    assert L["gated_scan_step"](*scan_step_args(B=0)) == OK
    assert L["act8_pack"](*pack_args(rows=0)) == OK
    assert L["act8_unpack"](*unpack_args(rows=0)) == OK


def test_workspace_sizes(L):
    n = ctypes.c_ulonglong()
    for N, T, C, packed in ((1, 1, 1, 0), (8, 4096, 2560, 0), (5, 12345, 333, 1), (0, 0, 7, 0), (3, 1 << 20, 64, 1)):
        assert L["gated_scan_grad_workspace_size"](N, T, C, packed, ctypes.byref(n)) == OK
        assert n.value < (64 << 20)
        for K in (1, 4, 8):
            assert L["conv_causal_grad_workspace_size"](N, T, C, K, packed, ctypes.byref(n)) == OK
            assert 4 * C * (K + 1) <= n.value < (64 << 20)
    assert L["gated_scan_grad_workspace_size"](1, 1, 0, 0, ctypes.byref(n)) == EINVAL
    assert L["conv_causal_grad_workspace_size"](1, 1, 1, 9, 0, ctypes.byref(n)) == EINVAL
    assert L["conv_causal_grad_workspace_size"](1, 1, 1, 1, 0, None) == EINVAL


def test_binding_refuses():
    import implicit_gemm_convolution_conv2d_b200 as cf
    x, w, d = torch.zeros(2, 5, 8), torch.zeros(8, 4), torch.zeros(8)
    for call in (lambda: cf.conv_causal(x, w), lambda: cf.conv_causal_grad(x, w, x), lambda: cf.conv_causal_step(x[0], w, torch.zeros(5, 3, 8)),
                 lambda: cf.gated_scan(x, x, x, d), lambda: cf.gated_scan_grad(x, x, x, d, x, torch.zeros(2, 1, 8)),
                 lambda: cf.gated_scan_step(x[0], x[0], x[0], d, torch.zeros(5, 8)), lambda: cf.act8_pack(x),
                 lambda: cf.act8_unpack(cf.Act8(torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4, 1, dtype=torch.uint8), torch.float32)),
                 lambda: cf.conv_wgrad(cf.Act8(torch.zeros(1, 4, 4, 8, dtype=torch.int8), torch.zeros(1, 4, 4, 1, dtype=torch.uint8),
                                               torch.float32), torch.zeros(1, 4, 4, 8), 3, padding=1)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        cf.act8_unpack(x)


# ---- the reference itself -----------------------------------------------


def test_reference_convolution_is_torchs():
    torch.manual_seed(0)
    x, w, b = torch.randn(2, 19, 6).double(), torch.randn(6, 4).double(), torch.randn(6).double()
    y = R.conv_causal(x, w, b, False, None, None)[0]
    z = torch.nn.functional.conv1d(torch.nn.functional.pad(x.transpose(1, 2), (3, 0)), w[:, None], b, groups=6).transpose(1, 2)
    assert torch.allclose(y, z, rtol=1e-13, atol=1e-13)
    packed = R.conv_causal(torch.cat([x[0], x[1, :7]]), w, b, True, None, torch.tensor([0, 19, 19, 26]))[0]
    assert torch.allclose(packed[:19], torch.nn.functional.silu(z[0])) and torch.allclose(packed[19:], torch.nn.functional.silu(z[1, :7]))


def test_reference_scan_by_its_closed_form():
    """With constant gates h[t] is a geometric sum."""
    x, one = torch.ones(1, 20, 1).double(), torch.zeros(1, 20, 1).double()
    decay = torch.tensor([0.3]).double()
    y, last = R.gated_scan(x, one, one, decay, torch.tensor([[2.0]]).double(), None)
    a = torch.exp(-decay / 2)
    t = torch.arange(1, 21).double()
    ref = a ** t * 2 + torch.sqrt(1 - a * a) * 0.5 * (1 - a ** t) / (1 - a)
    assert torch.allclose(y[0, :, 0], ref, rtol=1e-12) and torch.allclose(last[0], ref[-1:], rtol=1e-12)


def test_reference_gradients_are_differences():
    torch.manual_seed(1)
    cu = torch.tensor([0, 3, 3, 9])
    x, r, i = (torch.randn(10, 2).double().requires_grad_() for _ in range(3))
    decay, h0 = torch.rand(2).double().requires_grad_(), torch.randn(3, 2).double().requires_grad_()
    assert torch.autograd.gradcheck(lambda *a: R.gated_scan(*a, cu), (x, r, i, decay, h0))
    w, b, st = torch.randn(2, 4).double().requires_grad_(), torch.randn(2).double().requires_grad_(), torch.randn(3, 3, 2).double().requires_grad_()
    assert torch.autograd.gradcheck(lambda x, w, b, s: R.conv_causal(x, w, b, True, s, cu)[:2], (x, w, b, st))


def test_reference_checkpoint():
    torch.manual_seed(2)
    for dtype in (torch.float32, torch.float16, torch.bfloat16):
        x = (torch.randn(50, 70) * torch.exp2(torch.randint(-9, 10, (50, 1)).float())).to(dtype)
        q, s = R.act8(x)
        v = R.act8_values(q, s)
        step = torch.exp2(s.double() - 127).repeat_interleave(32, -1)[:, :70]
        assert ((v - x.double()).abs() <= step / 2).all()
        amax = x.double().abs()[:, :32].amax(1)
        assert (amax <= 127 * step[:, 0]).all() and (amax > 63.5 * step[:, 0]).all()


def test_planted_mistakes_are_caught():
    """The bounds are narrow enough to see a mistake: in each, something small is wrong with the result."""
    torch.manual_seed(3)
    x, r, i = (torch.randn(1, 60, 4).double() for _ in range(3))
    decay = torch.tensor([0.002, 0.05, 0.6, 3.0]).double()
    y, last = R.gated_scan(x, r, i, decay, None, None)
    b = R.scan_bounds(x, r, i, decay, None, None)
    for dtype in (torch.float32, torch.bfloat16):
        good = y.to(dtype)
        assert R.worst(good, y, b["y"], dtype) <= 1
        for bad in (R.gated_scan(x, r, i, decay * 1.01, None, None)[0], R.gated_scan(x * 1.02, r, i, decay, None, None)[0],
                    torch.roll(y, 1, 1), R.gated_scan(x, r, i + 0.05, decay, None, None)[0]):
            assert R.worst(bad.to(dtype), y, b["y"], dtype) > 1
    w, bias = torch.randn(4, 4).double(), torch.randn(4).double()
    y, _, z, S = R.conv_causal(x, w, bias, True, None, None)
    lim = R.conv_bound(z, S, 4, True)
    assert R.worst(y.bfloat16(), y, lim, torch.bfloat16) <= 1
    for bad in (R.conv_causal(x, w.flip(1), bias, True, None, None)[0], R.conv_causal(x, w, bias * 1.05, True, None, None)[0],
                R.conv_causal(x, w, bias, False, None, None)[0]):
        assert R.worst(bad.bfloat16(), y, lim, torch.bfloat16) > 1

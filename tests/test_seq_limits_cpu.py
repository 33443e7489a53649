"""Limits of the sequence operators' sizes, and their first use, without a GPU."""
from __future__ import annotations

import pytest
import torch


@pytest.fixture
def seq(monkeypatch):
    from implicit_gemm_convolution_conv2d_b200 import seq as mod
    monkeypatch.setattr(mod, "_cuda", lambda t, name, what: None)  # sizes without memory: meta tensors
    return mod


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


def test_sizes_past_32_bits_are_refused(seq):
    """The library takes sequences, rows of a step, slots and channels as 32-bit integers: more are refused, not cut off."""
    big, w = 2 ** 32 + 3, meta(8, 4)
    f32 = torch.float32
    many, wide, cu = meta(big, 1, 8), meta(1, 1, big), meta(big + 1, dtype=torch.int32)
    step, index = meta(big, 8), meta(big, dtype=torch.int32)
    calls = [
        lambda: seq.conv_causal(many, w),
        lambda: seq.conv_causal(wide, meta(big, 4)),
        lambda: seq.conv_causal(meta(5, 8), w, cu_seqlens=cu),
        lambda: seq.conv_causal_grad(many, w, many),
        lambda: seq.conv_causal_step(step, w, meta(4, 3, 8), index=index),
        lambda: seq.conv_causal_step(meta(2, 8), w, meta(big, 3, 8), index=meta(2, dtype=torch.int32)),
        lambda: seq.conv_causal_step(meta(1, big), meta(big, 4), meta(4, 3, big)),
        lambda: seq.gated_scan(many, many, many, meta(8, dtype=f32)),
        lambda: seq.gated_scan(wide, wide, wide, meta(big, dtype=f32)),
        lambda: seq.gated_scan_grad(many, many, many, meta(8, dtype=f32), many, meta(big, 1, 8, dtype=f32)),
        lambda: seq.gated_scan_step(step, step, step, meta(8, dtype=f32), meta(4, 8, dtype=f32), index=index),
        lambda: seq.gated_scan_step(meta(2, 8), meta(2, 8), meta(2, 8), meta(8, dtype=f32), meta(big, 8, dtype=f32)),
        lambda: seq.act8_pack(meta(2 ** 32 + 32)),
        lambda: seq.act8_pack(meta(1, 2 ** 32 + 32)),
        lambda: seq.act8_unpack(seq.Act8(meta(2 ** 32 + 32, dtype=torch.int8), meta(2 ** 27 + 1, dtype=torch.uint8), f32)),
    ]
    for k, call in enumerate(calls):
        with pytest.raises(ValueError, match=r"2\^31"):
            call()
            pytest.fail(f"call {k} was not refused")


# ---- the library --------------------------------------------------------


@pytest.fixture(scope="module")
def T():
    import tests.test_seq_cpu as T
    return T


@pytest.fixture(scope="module")
def lib():
    from implicit_gemm_convolution_conv2d_b200 import _build, seq
    _build.build()
    return seq._lib()


TOP = 2 ** 31 - 4096  # the first number that is refused


def test_last_channels_and_sequences_are_refused(lib, T):
    """Places behind the last channel or sequence fit 32 bits; C and N that they would not fit are refused (one row, one
    token or none, so that nothing else is too large)."""
    for C in (TOP, 2 ** 31 - 1):
        one = dict(N=1, L=1, C=C, cu=None)
        step = dict(B=1, slots=1, C=C, index=None)
        assert lib["conv_causal"](*T.conv_args(**one, K=1, state=None, state_out=None, y=1 << 40, w=1 << 50, bias=None)) == T.EINVAL
        assert lib["conv_causal_grad"](*T.conv_grad_args(**one, K=1, state=None, ds=None, dso=None, bias=None, db=None, w=1 << 50, dy=1 << 51,
                                                         dx=1 << 52, dw=1 << 53, ws=1 << 54, wb=1 << 40)) == T.EINVAL
        assert lib["conv_causal_step"](*T.conv_step_args(**step, K=1, bias=None, w=1 << 50, y=1 << 51)) == T.EINVAL
        assert lib["gated_scan"](*T.scan_args(**one, x=1 << 50, r=1 << 51, i=1 << 52, decay=1 << 53, h0=None, y=1 << 54, last=None,
                                              states=None)) == T.EINVAL
        assert lib["gated_scan_step"](*T.scan_step_args(**step, x=1 << 50, r=1 << 51, i=1 << 52, decay=1 << 53, h=1 << 54, y=1 << 55)) == T.EINVAL
        assert lib["act8_pack"](*T.pack_args(rows=1, C=C, q=1 << 50, scale=1 << 51)) == T.EINVAL
        assert lib["act8_unpack"](*T.unpack_args(rows=1, C=C, scale=1 << 50, y=1 << 51)) == T.EINVAL
        n = T.ctypes.c_ulonglong()
        assert lib["conv_causal_grad_workspace_size"](1, 1, C, 1, 0, T.ctypes.byref(n)) == T.EINVAL
        assert lib["gated_scan_grad_workspace_size"](1, 1, C, 0, T.ctypes.byref(n)) == T.EINVAL
    for N in (TOP, 2 ** 31 - 1):
        for L, cu in ((0, None), (5, 1 << 55)):
            assert lib["conv_causal"](*T.conv_args(N=N, L=L, C=1, K=1, cu=cu, xb=0, xt=1, state=None, state_out=None, bias=None)) == T.EINVAL
            assert lib["gated_scan"](*T.scan_args(N=N, L=L, C=1, cu=cu, xb=0, rb=0, ib=0, h0=None, last=1 << 50, states=None)) == T.EINVAL


def test_steps_refuse_channels_past_their_grid(lib, T):
    """A step's channels lie along a grid dimension of 65535 blocks: more are refused before a launch that would fail."""
    EUNSUPPORTED = -7
    far = dict(y=1 << 50, w=1 << 51, state=1 << 52)
    for C in (65535 * 128 + 1, 4 * 65535 * 128 + 4):
        assert lib["conv_causal_step"](*T.conv_step_args(B=1, C=C, K=2, bias=None, xt=C, **far)) == EUNSUPPORTED
        assert lib["gated_scan_step"](*T.scan_step_args(B=1, C=C, x=1 << 50, r=1 << 51, i=1 << 52, decay=1 << 53, h=1 << 54, y=1 << 55, xt=C,
                                                        rt=C, it=C)) == EUNSUPPORTED


# ---- first use ----------------------------------------------------------


def test_first_use_from_two_threads(monkeypatch):
    """A thread that comes while another one looks the functions up finds all of them."""
    import threading
    import types

    from implicit_gemm_convolution_conv2d_b200 import seq
    found = {}

    class Library:
        def __getattr__(self, name):
            if name == "gated_scan" and not found and threading.current_thread() is threading.main_thread():
                found["..."] = None
                other = threading.Thread(target=lambda: found.update(seq._lib()))
                other.start()
                other.join()
            return types.SimpleNamespace()

    library = Library()
    monkeypatch.setattr(seq, "_load", lambda: library)
    monkeypatch.setattr(seq, "_fn", {})
    mine = seq._lib()
    assert len(mine) == 10 and set(found) == set(mine) | {"..."}


def test_convolutions_alone_load_no_sequence_operators():
    """conv_wgrad of tensors looks for no checkpoint class."""
    import os
    import subprocess
    import sys

    code = ("import sys, torch, implicit_gemm_convolution_conv2d_b200 as cf\n"
            "try:\n    cf.conv_wgrad(torch.zeros(1, 4, 4, 8), torch.zeros(1, 4, 4, 8), 3, padding=1)\n"
            "except ValueError as e:\n    assert 'CUDA' in str(e)\n"
            "assert cf.__name__ + '.seq' not in sys.modules\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr

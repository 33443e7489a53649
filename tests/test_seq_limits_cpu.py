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

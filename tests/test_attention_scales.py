"""Scales that the attention operators refuse: scale * log2 e has to be a number of FP32.  No GPU; the fake pointers are never
dereferenced (sizes of 0 stand in for the accepted ones)."""
import pytest

from test_attention_args import attention, lib, prompt  # noqa: F401

MAX = 3.4028234663852886e38


@pytest.mark.parametrize("f", [prompt, attention])
@pytest.mark.parametrize("scale,status", [(MAX, 1), (-MAX, 1), (2.4e38, 1), (-2.4e38, 1), (2.3e38, 0), (-2.3e38, 0), (0.0, 0), (1e-45, 0)])
def test_scales(lib, f, scale, status):  # noqa: F811
    assert f(lib, scale=scale, Hq=0 if status == 0 else 4) == status

"""What the token path's binding makes of its arguments before any call (no GPU)."""
import struct

import pytest
import torch

from scan_linear_rnns_amd import tokens


@pytest.mark.parametrize("name, dtype, value, want", [
    ("top_k", torch.int32, -10 ** 12, "all"), ("top_k", torch.int32, -(1 << 31) - 1, "all"), ("top_k", torch.int32, 0, "all"),
    ("top_k", torch.int32, 10 ** 12, 2 ** 31 - 1), ("top_k", torch.int32, 7, 7),
    ("temperature", torch.float32, 1e39, float("inf")), ("temperature", torch.float32, -1e39, -float("inf")),
    ("temperature", torch.float32, 0.5, 0.5), ("temperature", torch.float32, 1, 1.0),
    ("top_p", torch.float32, 1e300, float("inf")), ("min_p", torch.float32, 1e300, float("inf")),
    ("min_p", torch.float32, float("nan"), "nan")])
def test_a_number_past_its_types_range(name, dtype, value, want):
    """It goes to the library as the definition takes it (0 or less: all; above 1: 1), not as an error of packing it."""
    off = 0 if name == "top_k" else 1.0
    got, ptr = tokens._setting(torch, name, value, dtype, 3, 0, off)
    assert ptr is None
    numbers = dict(top_k=0, temperature=1.0, top_p=1.0, min_p=0.0)
    numbers[name] = got
    packed = tokens._pack_sample(3, 10, 10, 0, *(numbers[n] for n in ("top_k", "temperature", "top_p", "min_p")))
    sent = struct.unpack("3q2i3f4x", packed)[4 + ("top_k", "temperature", "top_p", "min_p").index(name)]
    assert sent <= 0 if want == "all" else sent != sent if want == "nan" else sent == want

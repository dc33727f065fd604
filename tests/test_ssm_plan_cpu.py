"""Into how many segments of time the forward scan splits a call, read from its workspace (no GPU)."""
import os

import pytest

import linear_attention_recurrence_delta_gb300 as gdn


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(gdn.LIB_PATH):
        from linear_attention_recurrence_delta_gb300 import _build
        _build.build()
    return gdn.load()


def segments(B, T, D):
    """A state of 16 values and a sum for each of D channels (a multiple of 32) at B T / (tokens of a segment) + B places."""
    places = (gdn.gdn_scan_workspace_bytes(gdn.make_scan(B, T, D, 16), 0) - 256) / (D * 17 * 4)
    length = B * T / (places - B)
    return T / length


# warps of 32 channels, 16 an SM run at once: 152 x 16 / (B D / 32) segments are a round of them
@pytest.mark.parametrize("B,T,D", [(4, 2048, 4864), (1, 2048, 19456), (16, 1024, 1184), (1, 4096, 9376), (1, 4096, 6208)])
def test_few_segments_run_in_two_rounds(B, T, D):
    """One round of 4 to 12 segments is slower than two of twice as many (329 us and 300 for 4 x 2048 tokens of 4864 channels)."""
    round_ = 152 * 16 * 32 / (B * D)
    assert 4 <= round_ < 15
    assert abs(segments(B, T, D) - 2 * round_) <= 0.15 * 2 * round_


@pytest.mark.parametrize("B,T,D", [(8, 2048, 608), (1, 8192, 4096), (2, 4096, 2560), (1, 16000, 1536)])
def test_many_segments_run_in_one(B, T, D):
    round_ = 152 * 16 * 32 / (B * D)
    assert round_ >= 15
    assert abs(segments(B, T, D) - round_) <= 0.15 * round_

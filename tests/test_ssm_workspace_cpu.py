"""Sizes of the state-space operators' workspaces against what has to lie in them (no GPU)."""
import os

import pytest

import linear_attention_recurrence_delta_gb300 as gdn

MOST = 2**31 - 1      # T of a caller who knows no bound


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(gdn.LIB_PATH):
        from linear_attention_recurrence_delta_gb300 import _build
        _build.build()
    return gdn.load()


@pytest.mark.parametrize("B,D,W", [(1, 8, 4), (3, 64, 2), (700, 2048, 3), (65535, 1024, 4)])
@pytest.mark.parametrize("rows", [0, 1, 1000, 1 << 20])
def test_convolution_whatever_the_bound(B, D, W, rows):
    """No sequence is longer than the tensors, so a T past them asks for what T = rows does: rows of D (W + 1) sums, one for each block of
    a grid that is at most 152 x 32 blocks and at most a block for each 128 rows of a sequence."""
    need = [gdn.gdn_conv_workspace_bytes(gdn.make_conv(B, T, D, W, rows=rows)) for T in (max(rows, 1), rows + 12345, MOST - 127, MOST - 126, MOST)]
    assert len(set(need)) == 1
    blocks = min(152 * 32, B * max(1, -(-rows // 128)))
    assert 256 + D * (W + 1) * 4 <= need[0] <= 512 + blocks * D * (W + 1) * 4


@pytest.mark.parametrize("backward", [0, 1])
@pytest.mark.parametrize("rows", [0, 1, 1000, 1 << 20])
def test_scan_whatever_the_bound(rows, backward):
    need = [gdn.gdn_scan_workspace_bytes(gdn.make_scan(3, T, 64, 16, rows=rows), backward) for T in (max(rows, 1), MOST - 7, MOST)]
    assert len(set(need)) == 1 and need[0] >= 256


@pytest.mark.parametrize("B,T,D,N,G", [(4, 1000, 64, 16, 1), (1, 1, 8, 8, 1), (9, 333, 208, 8, 2), (2, 77, 96, 40, 3), (3, 8, 16, 64, 2)])
def test_scan_holds_what_it_keeps(B, T, D, N, G):
    """A state for every eighth token of each sequence; in the gradients' workspace a row of dA_log, dD and d dt_bias for each sequence and a
    row of dB and dC for each token, in the forward's of a split call the segments' states."""
    s = gdn.make_scan(B, T, D, N, G)
    state, rows = D * N * 4, B * T
    assert gdn.gdn_scan_saved_bytes(s) >= (rows // 8 + B) * state
    back = gdn.gdn_scan_workspace_bytes(s, 1)
    assert back >= B * D * (N + 2) * 4 + rows * G * 2 * N * 4 and back >= gdn.gdn_scan_workspace_bytes(s, 0)
    if T >= 128:      # few channels: at least four segments forwards
        assert gdn.gdn_scan_workspace_bytes(s, 0) >= 4 * B * state

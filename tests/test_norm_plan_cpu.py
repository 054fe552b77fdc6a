"""How many rows of tokens the group norm's backward pass takes at once, from its workspace (no GPU needed)."""
import os

import pytest
import torch

from state_space_sequence_chunk_amd import ssd

pytestmark = pytest.mark.skipif(not os.path.exists(ssd.LIB_PATH), reason="HIP library not built")


def rows(tokens, channels, groups):
    n = ssd.group_norm_backward_workspace_bytes(ssd.make_norm_shape(tokens, channels, groups, torch.float32))
    return n // 2 // (4 * channels)


@pytest.mark.parametrize("tokens,channels,groups,want", [
    # few channels a thread: four workgroups a compute unit (two took 1.4 to 1.7 times as long)
    (16000, 1024, 1, 1024), (8000, 1683, 9, 4 * (1024 // 9)), (16000, 999, 3, 2 * (1024 // 3)), (9000, 8192, 64, 128),
    # twelve: three (two and four took 1.1 to 1.3 times as long)
    (16000, 2700, 1, 768),
    # twenty: two (four took 1.04 to 1.12 times as long)
    (16384, 5120, 8, 512), (1024, 5120, 1, 512)])
def test_workgroups_a_compute_unit(tokens, channels, groups, want):
    assert rows(tokens, channels, groups) == want

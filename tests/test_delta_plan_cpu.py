"""Plans of the gated delta rule's kernels, from the library's host-only queries (no GPU needed)."""
import ctypes
import os
import re

import pytest

from state_space_sequence_chunk_amd import ssd

pytestmark = pytest.mark.skipif(not os.path.exists(ssd.LIB_PATH), reason="HIP library not built")


def shape(batch, seqlen, nheads, headdim, dstate, ngroups=1, dtype=ssd.SSD_BF16):
    return ssd.make_shape(batch, seqlen, nheads, headdim, dstate, ngroups, 64, dtype, ssd.SSD_F32)


def segments(s):
    """The forward walk's segments, from what its workspace holds beside each chunk's scalars and two
    matrices: the states entering all segments, and the first walk's rows for all but the last."""
    up = lambda n: -(-n // 256) * 256  # noqa: E731
    heads, P, S = s.batch * s.nheads, s.headdim, s.dstate
    chunks = heads * (-(-s.seqlen // 64))
    extra = ssd.delta_forward_workspace_bytes(s) - up(chunks * 5 * 64 * 4) - 2 * up(chunks * 6 * 2048)
    fits = [n for n in range(2, 17) if up(4 * heads * (n - 1) * (P + S) * S) + up(4 * heads * n * P * S) == extra]
    return fits[0] if extra else 1


@pytest.mark.parametrize("nheads,headdim,dstate,most", [(32, 16, 256, 1), (48, 16, 256, 1), (48, 16, 128, 3), (96, 16, 256, 1)])
def test_few_segments_where_the_first_walk_costs_more_than_it_saves(nheads, headdim, dstate, most):
    # a first walk carries headdim + dstate rows; five segments of 32 and 48 heads of 16 x 256 measured 1.25 and
    # 1.46 times one walk's time; 48 heads of 16 x 128: 1.16 in five segments, 0.93 in three
    assert segments(shape(1, 16384, nheads, headdim, dstate)) <= most


@pytest.mark.parametrize("s", [shape(4, 16384, 8, 64, 128), shape(1, 16384, 4, 16, 32), shape(1, 16384, 16, 128, 128),
                               shape(1, 16384, 16, 64, 256, dtype=ssd.SSD_F32), shape(2, 2048, 24, 64, 64, dtype=ssd.SSD_F32)])
def test_segments_where_they_pay(s):
    # 0.2 to 0.8 times one walk's time
    assert segments(s) > 1


@pytest.mark.parametrize("batch,seqlen,nheads,headdim,dstate,dtype,loop", [
    (96, 16, 32, 128, 256, ssd.SSD_BF16, False), (96, 24, 32, 128, 256, ssd.SSD_F32, False), (32, 16, 32, 64, 128, ssd.SSD_BF16, False),
    (96, 24, 32, 16, 16, ssd.SSD_BF16, True), (1, 32, 2, 128, 256, ssd.SSD_F32, True), (2, 16, 80, 64, 128, ssd.SSD_BF16, True),
    (96, 1, 32, 128, 256, ssd.SSD_BF16, True), (1, 65, 1, 16, 16, ssd.SSD_F32, False)])
def test_token_by_token_where_it_is_faster(batch, seqlen, nheads, headdim, dstate, dtype, loop):
    # 948 us token by token and 353 by chunks (first), 1413 and 724, 77 and 38; 30 and 53, 22 and 47, 19 and 21
    s = shape(batch, seqlen, nheads, headdim, dstate, dtype=dtype)
    assert (ssd.delta_forward_workspace_bytes(s) == 0) == loop


def test_plans():
    # the 2.7B layer: four waves a workgroup, ten of the group's 80 heads prepared by a wave, 40 a workgroup's gradients
    big = shape(2, 16384, 80, 64, 128)
    assert ssd.delta_forward_plan(big) == (1, 4, 0, 10) and ssd.delta_backward_plan(big) == (4, 10, 40)
    assert ssd.delta_backward_plan(shape(4, 4096, 48, 64, 128)) == (4, 3, 12)
    # few rows: a workgroup each
    assert ssd.delta_forward_plan(shape(1, 100, 2, 64, 64)) == (1, 1, 0, 1)
    assert ssd.delta_backward_plan(shape(1, 100, 2, 64, 64)) == (1, 1, 1)
    # no chunked kernel: token by token, or nothing
    assert ssd.delta_forward_plan(shape(2, 16, 80, 64, 128)) == (0, 0, 0, 0)
    assert ssd.delta_backward_plan(shape(2, 16, 80, 64, 128)) == (4, 1, 1)
    assert ssd.delta_forward_plan(shape(2, 0, 8, 64, 128)) == (0, 0, 0, 0)
    assert ssd.delta_backward_plan(shape(2, 0, 8, 64, 128)) == (0, 0, 0)
    for s in (shape(4, 16384, 8, 64, 128), shape(1, 4099, 24, 64, 64)):
        assert ssd.delta_forward_plan(s)[0] == segments(s) > 1
    lib = ssd.load_library()
    assert lib.ssd_delta_forward_plan(ctypes.byref(big), None, None, None, None) == 0
    assert lib.ssd_delta_backward_plan(ctypes.byref(big), None, None, None) == 0
    assert lib.ssd_delta_forward_plan(ctypes.byref(shape(2, 100, 8, 48, 128)), None, None, None, None) == 4
    assert lib.ssd_delta_backward_plan(None, None, None, None) == 1


ASM = os.path.join(os.path.dirname(ssd.LIB_PATH), "..", "_build", "k_delta_grads_f32.hip.s")


@pytest.mark.skipif(not os.path.exists(ASM), reason="no kernel assembly (written by the build)")
@pytest.mark.parametrize("headdim", [32, 64])
def test_gradients_at_dstate_256_take_all_registers(headdim):
    # held to half of them these instances of the fp32 gradients' kernel kept more than 2100 bytes a lane in scratch
    # memory and made the backward pass 15 to 25% slower
    text = open(ASM).read()
    name = f"delta_grads_kernelIfLi256ELi{headdim}EE"
    entry = [k for k in text[text.index("amdhsa.kernels:"):].split("  - .agpr_count:")[1:] if name in k]
    assert len(entry) == 1
    assert int(re.search(r"\.private_segment_fixed_size: (\d+)", entry[0]).group(1)) < 1024

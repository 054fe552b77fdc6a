"""Where the tensors and streams of a call lie: the binding refuses what a kernel could not
reach, before anything is enqueued (no GPU needed)."""
import os
import types

import pytest
import torch

import delta_ref as ref
from state_space_sequence_chunk_amd import ssd

built = pytest.mark.skipif(not os.path.exists(ssd.LIB_PATH), reason="HIP library not built")


@built
def test_tensors_of_the_host_are_refused():
    """Valid arguments but for where they lie: refused before a kernel gets their addresses."""
    d = ref.draw(2, 20, 4, 16, 16, 2, "fp32", 1)
    ins = [d[n] for n in ("v", "g", "beta", "k", "q", "h0")]
    one = [t[:, 0].contiguous() for t in ins[:5]]
    x, w = torch.zeros(4, 48), torch.ones(48)
    ssd_in = [torch.zeros(1, 64, 2, 16), torch.ones(1, 64, 2), torch.ones(2), torch.zeros(1, 64, 1, 16),
              torch.zeros(1, 64, 1, 16), torch.ones(2), torch.zeros(1, 2, 16, 16)]
    stream = types.SimpleNamespace(cuda_stream=0, device=x.device)  # never used
    for call in (lambda: ssd.delta_forward(*ins, stream=stream), lambda: ssd.delta_decode_step(*one, d["h0"], stream=stream),
                 lambda: ssd.delta_backward(*ins, d["dy"], d["dfinal"], stream=stream),
                 lambda: ssd.group_norm(x, w, stream=stream), lambda: ssd.group_norm_backward(x, w, None, x, stream=stream),
                 lambda: ssd.forward(*ssd_in, chunk=64, stream=stream),
                 lambda: ssd.backward(*ssd_in, ssd_in[0], chunk=64, stream=stream)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_a_stream_of_another_device_is_refused():
    """A stand-in for a tensor of the first GPU, and a stream of the second one."""
    t = types.SimpleNamespace(is_cuda=True, device=torch.device("cuda", 0))
    stream = types.SimpleNamespace(cuda_stream=0, device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="stream"):
        ssd._run(lambda: pytest.fail("called"), stream, (t,))

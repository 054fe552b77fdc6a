"""Group norm at sizes whose workgroups take several tokens one after another backwards (the last turn
not full) and whose threads hold three or five vectors, against the 64-bit definition.

Tolerances (relative 2-norm), roundings taken as independent. A statistic sums at most 64 squares a
thread and ten levels of a tree: sqrt(74 / 6) 2^-24, of which r keeps half. The sigmoid is within 4 steps of
2^-24 for these gates, and some six products follow: sqrt(16 + 6 + 1) 2^-24 = 2.9e-7, at most three
times that for channels that lie far from the mean: 1e-6. A gradient takes the difference of three such terms,
and dw and db a sum of at most 64 turns and rows: 3e-6."""
import pytest
import torch

import delta_ref as ref
from gpu_common import dev, needs_gpu
from state_space_sequence_chunk_amd import ssd

pytestmark = [pytest.mark.gpu, needs_gpu]

TOL, GRAD_TOL = 1e-6, 3e-6
# tokens, channels, groups (backwards, in vectors of 4: vectors a thread, threads a group)
SIZES = [
    (2100, 1280, 2),   # 5 of 32, two groups a workgroup
    (1100, 5120, 1),   # 5 of 256: sums through LDS, used again each turn
    (2100, 384, 1),    # 3 of 32
    (2100, 768, 1),    # 3 of 64; forwards, in vectors of 8, 3 of 32
    (9001, 64, 1),     # 1 of 16, many turns
    (1001, 1683, 9),   # single channels, 3 of 64
    (2049, 516, 1),    # 5 of 32, threads that hold no channel
    (33000, 48, 3),    # 1 of 4: 64 groups' threads a workgroup
]


def _rows(tokens, channels, groups):
    """Partial rows of dw, from the workspace: as many tokens are taken at once."""
    n = ssd.group_norm_backward_workspace_bytes(ssd.make_norm_shape(tokens, channels, groups, torch.float32))
    return n // 2 // (4 * channels)


@pytest.mark.parametrize("act", ["silu", "gate_pre", "gate_post"])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_several_turns(size, act, dtype):
    tokens, channels, groups = size
    assert tokens > _rows(*size)
    gen = torch.Generator().manual_seed(tokens + channels)
    n = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    center, gate = act == "silu", act.startswith("gate")
    d = {"x": (1.5 * n(tokens, channels) + 0.3).to(dtype), "w": 1 + 0.2 * n(channels), "b": 0.1 * n(channels)}
    if gate:
        d["z"] = n(tokens, channels).to(dtype)
    dy = n(tokens, channels)
    e = {m: dev(t) for m, t in d.items()}
    opts = dict(z=e.get("z"), groups=groups, center=center, act=act)
    wide = {m: t.double().requires_grad_() for m, t in e.items()}
    want = ref.norm(wide["x"], wide["w"], wide["b"], wide.get("z"), groups, 1e-5, center, act)
    out = ssd.group_norm(e["x"], e["w"], e["b"], **opts)
    err = ref.rel(out, want.detach().cpu())
    print(f"out {err:.1e}", flush=True)
    assert err <= TOL
    back = ssd.group_norm_backward(e["x"], e["w"], e["b"], dev(dy), **opts)
    again = ssd.group_norm_backward(e["x"], e["w"], e["b"], dev(dy), **opts)
    for m, g in zip(wide, torch.autograd.grad((want * dev(dy).double()).sum(), list(wide.values()))):
        err = ref.rel(back["d" + m], g.cpu())
        print(f"d{m} {err:.1e}", flush=True)
        assert err <= GRAD_TOL, m
        assert torch.equal(back["d" + m], again["d" + m])

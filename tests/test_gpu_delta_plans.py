"""Gated delta rule at the plans of real layers, against its 64-bit definition: two and four waves
a workgroup, several heads a wave of the preparation and a workgroup of the gradients (split
evenly and not), segments walked by one to four waves. Each test asserts the plan it is for.

Many short sequences and 64-bit references on the GPU keep it quick. Tolerances (relative 2-norm) add up
the steps of tests/delta_ref.py as independent roundings: each of at most 8 products of up to 256
terms adds sqrt(256 / 6) 2^-24 in fp32, a split operand 2^-18 / sqrt(3) twice and the dropped
product of remainders 2^-18 / 3 (a remainder is at most 2^-9 of its value, a third of that
square on average); the solve doubles an error's norm on average.
fp32: 2 sqrt(8) 6.5 2^-24 = 2.2e-6; bf16: 2 sqrt(8) 2^-18 sqrt(2 / 3 + 1 / 9) = 1.9e-5. An fp32 path that
took split bf16 operands (3e-6 and more) would fail the first."""
import pytest
import torch

import delta_ref as ref
from gpu_common import dev, needs_gpu
from state_space_sequence_chunk_amd import ssd

pytestmark = [pytest.mark.gpu, needs_gpu]

TOL = {"fp32": 2.2e-6, "bf16": 1.9e-5}
INPUTS = ("v", "g", "beta", "k", "q", "h0")
# batch, seqlen, heads, P, S, groups; waves a workgroup of the walks, heads a wave prepares, most heads
# a workgroup takes the gradients of
CASES = [
    ((22, 70, 3, 64, 64, 1), (2, 1, 1)),
    ((44, 65, 3, 64, 128, 1), (4, 1, 1)),
    ((35, 130, 2, 128, 128, 2), (4, 1, 1)),
    ((140, 65, 1, 32, 256, 1), (2, 1, 1)),
    ((70, 65, 2, 64, 256, 1), (4, 1, 1)),
    ((130, 65, 6, 64, 32, 1), (4, 1, 2)),    # four parts: 1, 2, 1 and 2 heads
    ((260, 65, 4, 128, 64, 2), (4, 1, 2)),
    ((280, 65, 4, 64, 256, 1), (4, 1, 2)),
    ((1050, 65, 3, 16, 16, 1), (1, 1, 3)),
    ((1050, 40, 3, 64, 128, 1), (4, 1, 3)),
    ((350, 130, 12, 32, 16, 1), (2, 3, 12)),
]
# segments, waves of the walk for y, waves of the first walk
SEGMENTS = [
    ((1, 2100, 2, 64, 32, 1), (4, 1, 1)),
    ((1, 4099, 8, 128, 128, 1), (8, 2, 2)),
    ((1, 4099, 24, 32, 32, 2), (8, 2, 2)),
    ((1, 4099, 16, 128, 64, 1), (6, 4, 2)),
    ((1, 4099, 24, 64, 64, 1), (8, 4, 4)),
    ((1, 4099, 24, 128, 128, 8), (4, 4, 4)),
]

# whether the sequence runs token by token, in bf16 and fp32: by what both ways cost, up to 64 tokens
SHORT = [
    ((1, 33, 2, 16, 16, 1), (True, True)),
    ((1, 48, 2, 64, 256, 1), (False, True)),
    ((2, 64, 1, 16, 16, 1), (False, False)),
    ((96, 16, 32, 64, 128, 4), (False, True)),
    ((96, 7, 32, 16, 64, 2), (True, True)),
    ((40, 5, 16, 128, 256, 1), (True, True)),
]


def _problem(shape, dtype, seed, **kw):
    d = ref.draw(*shape, dtype, seed, **kw)
    return {n: dev(t) for n, t in d.items()}


def _shape(e):
    return ssd.delta_shape_of(e["v"], e["k"])


def _close(got, want, tol, what):
    err = ref.rel(got, want.cpu())
    print(f"{what}: {err:.2e} (bound {tol:.1e})", flush=True)
    assert torch.isfinite(got).all() and err <= tol, what


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shape,plan", CASES)
def test_forward(shape, plan, dtype):
    e = _problem(shape, dtype, sum(shape))
    assert ssd.delta_forward_plan(_shape(e)) == (1, plan[0], 0, plan[1])
    y, final = ssd.delta_forward(*[e[n] for n in INPUTS], scale=0.5)
    want_y, want_f, _ = ref.forward(e, 0.5)
    _close(y, want_y, TOL[dtype], "y")
    _close(final, want_f, TOL[dtype], "final")
    if dtype == "bf16":
        yb, fb = ssd.delta_forward(*[e[n] for n in INPUTS], scale=0.5, out_dtype=torch.bfloat16)
        assert torch.equal(fb, final) and torch.equal(yb, y.bfloat16())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shape,plan", CASES)
def test_backward(shape, plan, dtype):
    e = _problem(shape, dtype, sum(shape) + 1)
    assert ssd.delta_backward_plan(_shape(e)) == plan
    got = ssd.delta_backward(*[e[n] for n in INPUTS], e["dy"], e["dfinal"], scale=0.5)
    again = ssd.delta_backward(*[e[n] for n in INPUTS], e["dy"], e["dfinal"], scale=0.5)
    want = ref.backward(e, 0.5)
    for n in want:
        _close(got[n], want[n], TOL[dtype], n)
        assert torch.equal(got[n], again[n]), n


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shape,loop", SHORT)
def test_short_sequences(shape, loop, dtype):
    e = _problem(shape, dtype, sum(shape))
    assert (ssd.delta_forward_plan(_shape(e))[0] == 0) == loop[dtype == "fp32"]
    y, final = ssd.delta_forward(*[e[n] for n in INPUTS], scale=0.5)
    want_y, want_f, _ = ref.forward(e, 0.5)
    _close(y, want_y, TOL[dtype], "y")
    _close(final, want_f, TOL[dtype], "final")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shape,plan", SEGMENTS)
def test_forward_by_segments(shape, plan, dtype):
    e = _problem(shape, dtype, sum(shape), gmin=-0.02)  # a state that lasts from segment to segment
    assert ssd.delta_forward_plan(_shape(e))[:3] == plan
    y, final = ssd.delta_forward(*[e[n] for n in INPUTS])
    want_y, want_f, _ = ref.forward(e)
    _close(y, want_y, TOL[dtype], "y")
    _close(final, want_f, TOL[dtype], "final")


def test_nan_in_one_head_of_many():
    # a workgroup's gradients go head by head: what a head leaves in LDS does not reach the next
    shape = (1050, 65, 3, 16, 16, 1)
    e = _problem(shape, "bf16", 9)
    assert ssd.delta_backward_plan(_shape(e))[2] == 3
    args = lambda: [e[n] for n in INPUTS] + [e["dy"], e["dfinal"]]  # noqa: E731
    a = ssd.delta_backward(*args())
    e["v"][:, :, 1] = float("nan")
    b = ssd.delta_backward(*args())
    for n in ("dv", "dg", "dbeta"):
        assert torch.equal(a[n][:, :, [0, 2]], b[n][:, :, [0, 2]]), n
    assert torch.equal(a["dh0"][:, [0, 2]], b["dh0"][:, [0, 2]])
    assert torch.isnan(b["dk"]).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 1, 80, 64, 128, 1), (96, 1, 32, 128, 128, 16), (3, 1, 2, 16, 256, 2), (1, 1, 1, 16, 16, 1)])
def test_step(shape, dtype):
    # fp32 arithmetic for either type
    e = _problem(shape, dtype, sum(shape))
    want_y, want_f, _ = ref.forward(e, 2.0)
    y = ssd.delta_decode_step(*[e[n][:, 0].contiguous() for n in INPUTS[:5]], e["h0"], scale=2.0)
    _close(y, want_y[:, 0], TOL["fp32"], "y")
    _close(e["h0"], want_f, TOL["fp32"], "state")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_layer(dtype):
    """Delta rule and gated norm of each head's rows, and their gradients, with four waves a workgroup in the
    walks, two heads a workgroup of the gradients and several turns in the norm. The norm divides y's error by
    each row's own size, down to a tenth of the usual one; its gradient does so again, and that of the
    delta rule starts from it."""
    shape = (130, 65, 6, 64, 32, 1)
    e = _problem(shape, dtype, 77)
    b, L, h, P = shape[:4]
    assert ssd.delta_backward_plan(_shape(e)) == (4, 1, 2)
    gen = torch.Generator().manual_seed(78)
    z, w, dout = (dev(torch.randn(s, generator=gen)) for s in ((b, L, h * P), (h * P,), (b, L, h * P)))
    z = z.to(e["v"].dtype)
    opts = dict(z=z, groups=h, act="gate_post")
    y, final = ssd.delta_forward(*[e[n] for n in INPUTS])
    out = ssd.group_norm(y.flatten(2), w, **opts)
    back = ssd.group_norm_backward(y.flatten(2), w, None, dout, **opts)
    grads = ssd.delta_backward(*[e[n] for n in INPUTS], back["dx"].view(b, L, h, P), e["dfinal"])
    ry, rf, _ = ref.forward(e)
    leaves = [t.requires_grad_() for t in (ry.flatten(2), w.double(), z.double())]
    rout = ref.norm(leaves[0], leaves[1], None, leaves[2], h, 1e-5, False, "gate_post")
    dy, dw, dz = torch.autograd.grad((rout * dout.double()).sum(), leaves)
    tol = 10 * TOL[dtype]
    _close(out, rout.detach(), tol, "out")
    _close(final, rf, TOL[dtype], "final")
    _close(back["dw"], dw, tol, "dw")
    _close(back["dz"], dz, tol, "dz")
    want = ref.backward({**e, "dy": dy.view(b, L, h, P)})
    for n in want:
        _close(grads[n], want[n], 10 * tol, n)

"""Gates that decay to zero: nothing passes them, so their gradients are zero, each of them, whatever the other values."""
import pytest
import torch

import gated_ref as ref
from test_gpu_gated import BF16, DEV, F32, TOL, covered, make, run_backward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("closed", [float("-inf"), -1e30, -200.0, -110.0])
@pytest.mark.parametrize("opening", [False, True])
@pytest.mark.parametrize("lens", [None, [129, 0, 40, 131]])
@pytest.mark.parametrize("dtype,dk,dv", [(F32, 48, 80), (F32, 128, 128), (BF16, 64, 64), (BF16, 128, 128), (BF16, 24, 56)])
def test_gradient_of_a_closed_gate(dtype, dk, dv, lens, opening, closed):
    """`opening`: some gates are positive (no 128 tokens add up to 80).  Values of some size: what is left of a sum that
    should cancel grows with them."""
    x = make(81, dtype, 1, 3, 300, dk, dv, "mild", lens)
    for m in ("q", "k", "v", "do"):
        x[m] *= 30
    gen = torch.Generator().manual_seed(8)
    if opening:
        x["g"][(torch.rand(x["g"].shape, generator=gen) < 0.2).to(DEV)] = 0.25
    at = (torch.rand(x["g"].shape, generator=gen) < 0.1).to(DEV)
    x["g"][at] = closed
    dg = run_backward(x)[3]
    assert bool((dg[at] == 0).all()), float(dg[at].float().abs().max())
    want = ref.prefill_backward(x["q"], x["k"], x["v"], x["g"], x["S0"], x["do"], x["dS"], lens)
    assert ref.rel(covered(dg, lens), want[3]) <= TOL[dtype]

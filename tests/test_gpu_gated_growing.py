"""Positive gates, within what the header allows: a memory that grows before a valley and again behind it.  The state
before the valley and the gradient behind it are both large, their product by itself beyond float32, the decayed one not."""
import pytest

import gated_ref as ref
from test_gpu_gated import BF16, F32, TOL, TOL_STATE, make, run_backward, run_prefill

pytestmark = pytest.mark.gpu

# (tokens, gate): valleys that fill a chunk of 32 and one of 128; any 128 tokens hold positive gates of 78 and 66
HILLS = {"near": [(98, 128, 1.3), (128, 160, -2.5), (160, 190, 1.3)], "far": [(68, 128, 1.1), (128, 192, -1.1), (256, 316, 1.1)]}


@pytest.mark.parametrize("where", list(HILLS))
@pytest.mark.parametrize("dtype,dk,dv", [(F32, 48, 80), (F32, 128, 128), (BF16, 64, 64), (BF16, 128, 128), (BF16, 24, 56)])
def test_growth_and_valley(dtype, dk, dv, where):
    x = make(111, dtype, 1, 2, 400, dk, dv, "none")
    for m in ("q", "k", "v", "do"):
        x[m] *= 30
    for a, b, g in HILLS[where]:
        x["g"][:, :, a:b] = g
    args = [x[m] for m in ("q", "k", "v", "g")]
    got = [*run_prefill(x), *run_backward(x)]
    want = [*ref.prefill(*args, x["S0"]), *ref.prefill_backward(*args, x["S0"], x["do"], x["dS"])]
    for name, a, b in zip(("o", "S", "dq", "dk", "dv", "dg", "dS0"), got, want):
        err = ref.rel(a, b)
        assert err <= (TOL_STATE if name in ("S", "dS0") else TOL[dtype]), (name, err)


@pytest.mark.parametrize("dtype,dk,dv,T,rise", [(BF16, 64, 64, 2200, (640, 1280, 0.15)), (BF16, 128, 128, 2200, (640, 1280, 0.15)),
                                                (F32, 8, 8, 16384, (8192, 8448, 0.4))])
def test_growth_over_a_segment(dtype, dk, dv, T, rise):
    """A segment of the walk that grows by e^96 and e^102, and small values for it.  The exponents, up to 148 powers of two,
    are float32 sums on the tensor cores: 20 roundings of at most 2^-18 each put e^x at most 20 * 2^-18 * ln 2 < 2^-14 off."""
    x = make(112, dtype, 1, 2, T, dk, dv)
    for m in ("v", "do", "S0", "dS"):
        x[m] *= 1e-12
    a, b, g = rise
    x["g"][:, :, a:b] = g
    args = [x[m] for m in ("q", "k", "v", "g")]
    got = [*run_prefill(x), *run_backward(x)]
    want = [*ref.prefill(*args, x["S0"]), *ref.prefill_backward(*args, x["S0"], x["do"], x["dS"])]
    for name, u, w in zip(("o", "S", "dq", "dk", "dv", "dg", "dS0"), got, want):
        err = ref.rel(u, w)
        assert err <= (2 * TOL_STATE if name in ("S", "dS0") else TOL[dtype]), (name, err)

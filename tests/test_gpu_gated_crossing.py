"""What crosses a whole chunk in a gate's gradient, e^{G_C} <E, S>: one number for all of its tokens, in which large
products may cancel.  With q = k = 0 it is all there is: dg_t = e^{sum of all gates} <dS, S_0>.  Sequences of one chunk of
128 tokens, which is summed in float32 whatever the type."""
import numpy as np
import pytest
import torch

import gated_ref as ref
from test_gpu_gated import BF16, DEV, F32, make, run_backward

pytestmark = pytest.mark.gpu

LENGTHS = [1, 5, 32, 33, 127, 128]


def _check(x, T, lens, spread):
    """spread: of the 2-norm of the products E S, what the stored states may leave out; half a step of the result besides."""
    x["q"].zero_()
    x["k"].zero_()
    dg = ref.f64(run_backward(x)[3])[0]                       # [H, T]
    H, units = dg.shape[0], [(0, T)] if lens is None else [(sum(lens[:n]), sum(lens[:n + 1])) for n in range(len(lens))]
    g = ref.f64(x["g"])[0]
    for n, (a, b) in enumerate(units):
        for h in range(H):
            if a == b:
                continue
            E, S = (ref.f64(x[m])[n * H + h] for m in ("dS", "S0"))
            f = np.exp(g[h, a:b].sum())
            off = np.abs(dg[h, a:b] - f * (E * S).sum()).max()
            assert off <= 2.0 ** -8 * abs(f * (E * S).sum()) + spread * f * np.linalg.norm(E * S), (n, h, off)


@pytest.mark.parametrize("H", [2, 40])      # 32 units and more: other kernels
@pytest.mark.parametrize("T", LENGTHS)
@pytest.mark.parametrize("dtype,d", [(BF16, 64), (BF16, 128), (F32, 64)])
def test_states_that_bf16_does_not_tell_apart(dtype, d, T, H):
    """S_0 is 1 + 2^-9 where dS is 1 and 1 where it is -1: their product is 2^-9 for each pair, 0 after a rounding."""
    x = make(1, dtype, 1, H, T, d, d, "none")
    sign = torch.tensor([1.0, -1.0], device=DEV).repeat(d // 2)
    x["dS"] = sign.expand(H, d, d).contiguous()
    x["S0"] = 1 + 2.0 ** -9 * (x["dS"] > 0)
    _check(x, T, None, 0.0)


@pytest.mark.parametrize("lens", [None, [20, 1, 128, 0, 64, 65]])
@pytest.mark.parametrize("dtype,d", [(BF16, 64), (BF16, 128), (F32, 64)])
@pytest.mark.parametrize("T", [20, 100])
def test_states_of_random_signs(dtype, d, T, lens):
    """A thread adds 64 products in float32 and a tree those of 256: 72 roundings at most on any product's way, each 2^-24 of
    a partial sum, which stays within a few times the 2-norm of all products: less than 2^-13 of that."""
    T = T if lens is None else sum(lens)
    x = make(2, dtype, 1, 40, T, d, d, "mild", lens)
    x["g"] *= 0.1                                               # a long memory
    _check(x, T, lens, 2.0 ** -13)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,H", [([1], 1), ([0, 5], 1), ([3, 0, 2], 1), ([20, 12], 16), ([1, 1], 17), ([20, 13], 16)])
def test_short_packed_units(d, lens, H):
    err = norm = 0.0
    for seed in range(8):
        x = make(400 + seed, BF16, 1, H, sum(lens), d, d, "mild", lens)
        want = ref.prefill_backward(x["q"], x["k"], x["v"], x["g"], x["S0"], x["do"], x["dS"], lens)[3]
        err += np.linalg.norm(ref.f64(run_backward(x)[3]) - want) ** 2
        norm += np.linalg.norm(want) ** 2
    assert err <= 2.0 ** -16 * norm, (err / norm) ** 0.5


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,H", [(1, 1), (1, 2), (1, 33), (5, 1), (5, 33), (20, 1), (20, 33), (32, 3), (33, 3)])
def test_short_units(d, T, H):
    """As they come, eight times over.  A rounding is off by at most 2^-8, evenly spread, so by 2^-8 / sqrt(3) in the mean square:
    two of them, of an operand and of the result, by less than 2^-8."""
    err = norm = 0.0
    for seed in range(8):
        x = make(300 + seed, BF16, 1, H, T, d, d)
        want = ref.prefill_backward(x["q"], x["k"], x["v"], x["g"], x["S0"], x["do"], x["dS"])[3]
        err += np.linalg.norm(ref.f64(run_backward(x)[3]) - want) ** 2
        norm += np.linalg.norm(want) ** 2
    assert err <= 2.0 ** -16 * norm, (err / norm) ** 0.5

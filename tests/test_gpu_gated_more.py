"""More of the gated recurrence on the GPU: many packed sequences, what a state keeps, units of very different size, and
sequences beside one that is not finite."""
import numpy as np
import pytest
import torch

import gated_ref as ref
from test_gpu_gated import BF16, DEV, F32, TOL, TOL_STATE, check_backward, check_prefill, make, run_backward, run_prefill

pytestmark = pytest.mark.gpu

TYPES = [(F32, 20, 36), (BF16, 64, 64), (BF16, 128, 128)]


@pytest.mark.parametrize("n", [1023, 1024, 1025, 2048, 2500])
@pytest.mark.parametrize("dtype,dk,dv", TYPES)
def test_many_sequences(dtype, dk, dv, n):
    """Around the 1024 sequences that one pass over the offsets takes, and that are put in order: short and empty ones, one
    longer than a chunk early and one late."""
    lens = np.random.default_rng(n).integers(0, 4, n).tolist()
    lens[5], lens[-3] = 140, 270
    x = make(n, dtype, 1, 1, sum(lens) + 2, dk, dv, "mild", lens)
    check_prefill(x, dtype)
    check_backward(x, dtype)


@pytest.mark.parametrize("at", [0, 10, 98])
@pytest.mark.parametrize("d", [64, 128])
def test_what_a_state_keeps(d, at):
    """One token that is not zero and one gate: the final state is e^g k v^T, the gradient of the first e^g q do^T.  Of each
    element: 2^-22 by the exponential, 2^-24 by its argument and by each of the two splits into three bf16 numbers, and
    at most 2^-23 at each of the two additions of the three products: less than 2^-20."""
    gen = torch.Generator().manual_seed(d + at)
    B, H, T = 1, 2, 100
    x = {m: torch.zeros(B, H, T, d, dtype=BF16, device=DEV) for m in ("q", "k", "v", "do")}
    for t in x.values():
        t[:, :, at] = torch.randn(B, H, d, generator=gen).to(BF16).to(DEV)
    x["g"] = torch.zeros(B, H, T, dtype=BF16, device=DEV)
    x["g"][:, :, at + 1] = torch.tensor([-0.3, -1.1]).to(BF16).to(DEV)     # behind the token: the state decays by it
    x.update(S0=torch.zeros(H, d, d, device=DEV), dS=torch.zeros(H, d, d, device=DEV), cu=None, lens=None)
    _, S = run_prefill(x)
    a = np.exp(ref.f64(x["g"][0, :, at + 1]))[:, None, None]
    k, v, q, do = (ref.f64(x[m][0, :, at]) for m in ("k", "v", "q", "do"))
    want = a * k[:, :, None] * v[:, None, :]
    assert (np.abs(ref.f64(S) - want) <= 2.0 ** -20 * np.abs(want)).all()
    x["g"].zero_()
    x["g"][:, :, at] = torch.tensor([-0.3, -1.1]).to(BF16).to(DEV)         # on the token: the gradient passes it
    dS0 = run_backward(x)[4]
    want = a * q[:, :, None] * do[:, None, :]
    assert (np.abs(ref.f64(dS0) - want) <= 2.0 ** -20 * np.abs(want)).all()


@pytest.mark.parametrize("dtype,dk,dv", TYPES)
@pytest.mark.parametrize("T", [20, 300])
def test_units_of_different_size(dtype, dk, dv, T):
    """Each unit by itself, the values of one a thousandth of those of the one before."""
    x = make(101, dtype, 1, 4, T, dk, dv)
    scale = torch.tensor([1.0, 1e-3, 1e-6, 1e-9], device=DEV)
    for m in ("v", "do"):
        x[m] = (x[m] * scale[None, :, None, None]).to(dtype)
    for m in ("S0", "dS"):
        x[m] = x[m] * scale[:, None, None]
    args = [x[m] for m in ("q", "k", "v", "g")]
    got = [*run_prefill(x), *run_backward(x)]
    want = [*ref.prefill(*args, x["S0"]), *ref.prefill_backward(*args, x["S0"], x["do"], x["dS"])]
    for name, a, b in zip(("o", "S", "dq", "dk", "dv", "dg", "dS0"), got, want):
        tol = TOL_STATE if name in ("S", "dS0") else TOL[dtype]
        a, b = (np.asarray(ref.f64(t)).reshape(4, -1) for t in (a, b))
        for u in range(4):
            assert ref.rel(a[u], b[u]) <= tol, (name, u)


@pytest.mark.parametrize("dtype,dk,dv", TYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_sequence_that_is_not_finite_stays_alone(dtype, dk, dv, bad):
    """Its rows lie in the tiles of its neighbours."""
    lens = [100, 60, 100, 5]
    x = make(102, dtype, 1, 3, sum(lens), dk, dv, "mild", lens)
    y = {m: t.clone() if isinstance(t, torch.Tensor) else t for m, t in x.items()}
    for m in ("q", "k", "v", "do", "g"):
        y[m][:, :, 100:160] = bad
    for m in ("S0", "dS"):
        y[m][3:6] = bad
    rows = [*range(100), *range(160, 265)]
    for fn in (run_prefill, run_backward):
        *got, S = fn(y)
        *want, S2 = fn(x)
        assert all(torch.equal(a[:, :, rows], b[:, :, rows]) for a, b in zip(got, want))
        assert torch.equal(S[:3], S2[:3]) and torch.equal(S[6:], S2[6:])

"""The longest sequence that a call takes, 2^31 - 1 tokens, with heads of one element on the CUDA cores.

All values are small whole numbers whose running sums repeat every 37 tokens, so every sum is exact in float32."""
import pytest
import torch

import recurrent_decode_la_b200 as la

pytestmark = pytest.mark.gpu

T, P = (1 << 31) - 1, 37
DEV = "cuda"


def _by_place(values):
    """[1, 1, T, 1]: values[t % P] for every token t."""
    out = torch.empty(T, device=DEV)
    row = torch.tensor(values, dtype=torch.float32, device=DEV)
    whole = T // P * P
    out[:whole].view(-1, P).copy_(row)
    out[whole:].copy_(row[:T - whole])
    return out.view(1, 1, T, 1)


def _is_by_place(x, values):
    x, row = x.view(-1), torch.tensor(values, dtype=torch.float32, device=DEV)
    whole, step = T // P * P, P << 22
    return all(bool((x[a:min(a + step, whole)].view(-1, P) == row).all()) for a in range(0, whole, step)) and torch.equal(
        x[whole:], row[:T - whole])


@pytest.mark.parametrize("packed", [False, True])
def test_longest_sequence(packed):
    if torch.cuda.get_device_properties(0).total_memory < 100 << 30:
        pytest.skip("needs 60 GB")
    v = [1.0] * 18 + [-1.0] * 18 + [0.0]
    S = [sum(v[:t + 1]) for t in range(P)]                      # S_t
    last = S[(T - 1) % P]
    D = [last - S[t] + v[t] for t in range(P)]                  # the sum of the gradients of o_t .. o_T
    ones, vs = _by_place([1.0] * P), _by_place(v)
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV) if packed else None
    n = 1 if packed else 0

    def ws(size):
        return torch.full((size(torch.float32, 1, 1, T, 1, 1, n),), 0xFF, dtype=torch.uint8, device=DEV)

    o, state = torch.full_like(vs, float("nan")), torch.zeros(1, 1, 1, device=DEV)
    la.la_gated_prefill(ones, ones, vs, None, o, state, cu_seqlens=cu, workspace=ws(la.la_gated_prefill_workspace_size))
    assert la.la_device_status() == la.LA_OK
    assert float(state) == last and _is_by_place(o, S)
    dq, dk, dv = o.fill_(float("nan")), torch.full_like(vs, float("nan")), torch.full_like(vs, float("nan"))
    dstate = torch.zeros_like(state)
    la.la_gated_prefill_backward(ones, ones, vs, None, None, vs, dstate, dq, dk, dv, cu_seqlens=cu,
                                 workspace=ws(la.la_gated_prefill_backward_workspace_size))
    assert la.la_device_status() == la.LA_OK
    assert float(dstate) == D[0]
    assert _is_by_place(dq, [a * b for a, b in zip(S, v)])
    assert _is_by_place(dk, [a * b for a, b in zip(D, v)])
    assert _is_by_place(dv, D)

"""The hand-off of chunk states through the workspace: every call begins with a workspace of NaNs, so that a state which
is read before all of it is there shows in the outputs, in a second call as in the first."""
import pytest
import torch

import gated_ref as ref
import recurrent_decode_la_b200 as la
from test_gpu_gated import BF16, TOL, TOL_STATE, covered, make, run_backward, run_prefill, ws_for

pytestmark = pytest.mark.gpu

# many units, few in segments, packed ones with chunks of one token
CASES = {"many": (12, 16, 900, None), "few": (1, 3, 6000, None), "packed": (1, 16, 5000, [2600, 0, 1, 1400, 129, 870])}


def _same(got, want):
    return all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("d", [64, 128])
def test_prefills_at_once(d):
    """Three streams that share the device, twelve times."""
    xs = [make(50 + i, BF16, *c[:3], d, d, "mild", c[3]) for i, c in enumerate(CASES.values())]
    want = [[t.clone() for t in run_prefill(x)] for x in xs]
    ws = [ws_for(x, False) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(12):
        got = [(torch.empty_like(x["v"]), x["S0"].clone()) for x in xs]
        torch.cuda.synchronize()
        for x, w, s, (o, S) in zip(xs, ws, streams, got):
            with torch.cuda.stream(s):
                w.fill_(0xFF)
                la.la_gated_prefill(x["q"], x["k"], x["v"], x["g"], o, S, cu_seqlens=x["cu"], workspace=w)
        torch.cuda.synchronize()
        assert la.la_device_status() == la.LA_OK
        assert all(_same(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("case", list(CASES))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("backward", [False, True])
def test_replays(case, d, backward):
    """A captured call, its workspace filled by the graph, ten times."""
    B, H, T, lens = CASES[case]
    x = make(60, BF16, B, H, T, d, d, "mild", lens)
    want = [t.clone() for t in (run_backward if backward else run_prefill)(x)]
    ws = ws_for(x, backward)
    outs = [torch.empty_like(x[m]) for m in ("q", "k", "v", "g")] if backward else [torch.empty_like(x["v"])]
    st = torch.empty_like(x["S0"])

    def call():
        ws.fill_(0xFF)
        if backward:
            st.copy_(x["dS"])
            la.la_gated_prefill_backward(x["q"], x["k"], x["v"], x["g"], x["S0"], x["do"], st, *outs, cu_seqlens=x["cu"], workspace=ws)
        else:
            st.copy_(x["S0"])
            la.la_gated_prefill(x["q"], x["k"], x["v"], x["g"], *outs, st, cu_seqlens=x["cu"], workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(10):
        for t in (*outs, st):
            t.zero_()
        graph.replay()
        assert la.la_device_status() == la.LA_OK
        assert _same([*outs, st], want)


@pytest.mark.parametrize("d", [64, 128])
def test_long_walks(d):
    """4096 chunks a call, more than the device holds at once."""
    x = make(70, BF16, 4, 16, 8192, d, d)
    want = [t.clone() for t in run_prefill(x)]
    ws = ws_for(x, False)
    for _ in range(6):
        ws.fill_(0xFF)
        o, S = run_prefill(x, ws=ws)
        assert bool(torch.isfinite(o).all())
        assert _same((o, S), want)
        del o, S


EMPTY = {"one walk, then empty ones": [130] + [0] * 40, "few walks": [130, 0, 0, 1, 300] + [0] * 300 + [129],
         "in segments": [0] * 6 + [1400] + [0] * 2, "unordered": [5, 0, 130] + [0] * 1100 + [1, 200] + [0] * 50, "all empty": [0] * 30}


@pytest.mark.parametrize("case", list(EMPTY))
@pytest.mark.parametrize("d", [64, 128])
def test_empty_sequences(case, d):
    """Many more empty sequences than others: a CTA takes many in a row."""
    lens = EMPTY[case]
    T = max(sum(lens), 3)
    x = make(90, BF16, 1, 2, T, d, d, "mild", lens)
    o, S = run_prefill(x)
    some = [n for n, m in enumerate(lens) if m]
    want = x["S0"].view(len(lens), 2, d, d)
    if some:
        oo, SS = ref.prefill(x["q"], x["k"], x["v"], x["g"], want[some], [lens[n] for n in some])
        assert ref.rel(covered(o, lens), oo) <= TOL[BF16]
        assert ref.rel(S.view(len(lens), 2, d, d)[some], SS.reshape(-1, 2, d, d)) <= TOL_STATE
    none = [n for n, m in enumerate(lens) if not m]
    assert torch.equal(S.view(len(lens), 2, d, d)[none], want[none])

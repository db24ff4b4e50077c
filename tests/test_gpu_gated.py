"""The gated recurrence, its gradient and rotary positions on the GPU against the float64 definitions (gated_ref.py).

Errors are 2-norms relative to the reference.  Tolerances, derived before the first run:

* bf16 results: each rounding moves a value by at most half a step, 2^-8 of it.  A result is rounded once, and its two
  parts (through the state, inside the chunk) each have one operand rounded once more: at most 3 * 2^-8.
* float32 results of float32 inputs: sums of up to 128 + 128 products in order, each step at most 2^-24 of the partial
  sum, and the exponents of the decays, at most 16 * 2^-24 off: 2^-15 covers 512 such steps.
* float32 states of bf16 inputs: a weighted key is kept to at most 2^-16 of it, the sums are float32: 2^-15."""
import numpy as np
import pytest
import torch

import gated_ref as ref
import recurrent_decode_la_b200 as la

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TOL = {BF16: 3 * 2.0 ** -8, F32: 2.0 ** -15}
TOL_STATE = 2.0 ** -15
DEV = "cuda"


def gates(gen, shape, kind):
    x = torch.randn(shape, generator=gen)
    if kind == "mild":
        return torch.nn.functional.logsigmoid(x + 4)
    if kind == "strong":                      # a few tokens of memory
        return -3 * x.abs()
    if kind == "none":
        return torch.zeros(shape)
    if kind == "resets":                      # some gates start afresh
        g = torch.nn.functional.logsigmoid(x + 3)
        g[torch.rand(shape, generator=gen) < 0.05] = float("-inf")
        return g
    if kind == "closed":                      # every gate does
        return torch.full(shape, float("-inf"))
    return torch.where(x > 1, -200.0, -0.01 * x.abs())   # "cliff": finite gates whose decay underflows


def make(seed, dtype, B, H, T, dk, dv, kind="mild", lens=None):
    gen = torch.Generator().manual_seed(seed)
    n = (len(lens) if lens is not None else B) * H
    q = torch.randn(B, H, T, dk, generator=gen) / dk ** 0.5
    k = torch.nn.functional.normalize(torch.randn(B, H, T, dk, generator=gen), dim=-1)
    v, do = torch.randn(B, H, T, dv, generator=gen), torch.randn(B, H, T, dv, generator=gen)
    g = None if kind is None else gates(gen, (B, H, T), kind).to(dtype).to(DEV)
    S0, dS = (torch.randn(n, dk, dv, generator=gen).to(DEV) * 0.3 for _ in range(2))
    q, k, v, do = (x.to(dtype).to(DEV) for x in (q, k, v, do))
    cu = None
    if lens is not None:
        cu = torch.tensor([0, *np.cumsum(lens)], dtype=torch.int32, device=DEV)
    return dict(q=q, k=k, v=v, g=g, S0=S0, do=do, dS=dS, cu=cu, lens=lens)


def ws_for(x, backward):
    B, H, T, dk = x["q"].shape
    size = la.la_gated_prefill_backward_workspace_size if backward else la.la_gated_prefill_workspace_size
    n = size(x["q"].dtype, B, H, T, dk, x["v"].shape[-1], 0 if x["cu"] is None else x["cu"].numel() - 1)
    return torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)   # NaNs: nothing may come from the workspace unwritten


def run_prefill(x, ws=None, max_seqlen=0):
    o, S = torch.full_like(x["v"], float("nan")), x["S0"].clone()
    la.la_gated_prefill(x["q"], x["k"], x["v"], x["g"], o, S, cu_seqlens=x["cu"], max_seqlen=max_seqlen,
                        workspace=ws_for(x, False) if ws is None else ws)
    assert la.la_device_status() == la.LA_OK
    return o, S


def run_backward(x, ws=None, s0=True):
    out = {n: torch.full_like(x[m], float("nan")) for n, m in (("dq", "q"), ("dk", "k"), ("dv", "v"))}
    out["dg"] = torch.full(x["q"].shape[:3], float("nan"), dtype=x["q"].dtype, device=DEV)
    D = x["dS"].clone()
    la.la_gated_prefill_backward(x["q"], x["k"], x["v"], x["g"], x["S0"] if s0 else None, x["do"], D, out["dq"], out["dk"],
                                 out["dv"], out["dg"], cu_seqlens=x["cu"], workspace=ws_for(x, True) if ws is None else ws)
    assert la.la_device_status() == la.LA_OK
    return out["dq"], out["dk"], out["dv"], out["dg"], D


def covered(y, lens):
    """Rows that a sequence covers; the rows behind the last one must be as they were (NaN)."""
    if lens is None:
        return y
    n = int(sum(lens))
    assert torch.isnan(y[:, :, n:]).all()
    return y[:, :, :n]


def check_prefill(x, dtype, **kw):
    o, S = run_prefill(x, **kw)
    n = sum(x["lens"]) if x["lens"] is not None else x["q"].shape[2]
    cut = {m: x[m][:, :, :n] if x[m] is not None else None for m in ("q", "k", "v", "g")}
    oo, SS = ref.prefill(cut["q"], cut["k"], cut["v"], cut["g"], x["S0"], x["lens"])
    assert ref.rel(covered(o, x["lens"]), oo) <= TOL[dtype]
    assert ref.rel(S, SS) <= TOL_STATE


def check_backward(x, dtype, s0=True, **kw):
    got = run_backward(x, s0=s0, **kw)
    n = sum(x["lens"]) if x["lens"] is not None else x["q"].shape[2]
    cut = {m: x[m][:, :, :n] if x[m] is not None else None for m in ("q", "k", "v", "g", "do")}
    want = ref.prefill_backward(cut["q"], cut["k"], cut["v"], cut["g"], x["S0"] if s0 else 0 * x["S0"], cut["do"], x["dS"], x["lens"])
    for name, y, r in zip(("dq", "dk", "dv", "dg", "dS0"), got, want):
        err = ref.rel(y if name == "dS0" else covered(y, x["lens"]), r)
        assert err <= (TOL_STATE if name == "dS0" else TOL[dtype]), (name, err)


SHAPES = [(F32, 8, 8), (F32, 48, 80), (F32, 128, 128), (F32, 1, 7), (F32, 127, 33), (BF16, 64, 64), (BF16, 128, 128),
          (BF16, 96, 96), (BF16, 40, 128), (BF16, 5, 3)]


@pytest.mark.parametrize("T", [1, 2, 16, 17, 31, 33, 127, 128, 129, 300])
@pytest.mark.parametrize("dtype,dk,dv", SHAPES)
def test_dense(dtype, dk, dv, T):
    x = make(T, dtype, 2, 3, T, dk, dv)
    check_prefill(x, dtype)
    check_backward(x, dtype)


@pytest.mark.parametrize("kind", [None, "none", "strong", "resets", "closed", "cliff"])
@pytest.mark.parametrize("dtype,dk,dv", [(F32, 48, 80), (BF16, 64, 64), (BF16, 128, 128), (BF16, 24, 56)])
@pytest.mark.parametrize("T", [9, 200, 385])
def test_gates(dtype, dk, dv, kind, T):
    x = make(7, dtype, 1, 2, T, dk, dv, kind)
    check_prefill(x, dtype)
    check_backward(x, dtype)


PACKED = [[1], [0], [0, 0, 5], [300], [128, 128], [127, 1, 0, 129, 64], [1] * 20, [17, 250, 3, 0, 0, 140]]


@pytest.mark.parametrize("lens", PACKED, ids=str)
@pytest.mark.parametrize("dtype,dk,dv", [(F32, 48, 80), (BF16, 64, 64), (BF16, 128, 128), (BF16, 20, 36)])
@pytest.mark.parametrize("behind", [0, 5])
def test_packed(dtype, dk, dv, lens, behind):
    """Sequences of any length, and rows behind the last one, which hold NaN and stay as they are."""
    T = sum(lens) + behind
    if T == 0:
        T = 3
    x = make(11, dtype, 1, 3, T, dk, dv, "resets", lens)
    for m in ("q", "k", "v", "do", "g"):
        x[m][:, :, sum(lens):] = float("nan")
    check_prefill(x, dtype)
    check_backward(x, dtype)
    if max(lens) <= 16:
        check_prefill(x, dtype, max_seqlen=max(max(lens), 1))


@pytest.mark.parametrize("dtype,dk,dv", [(F32, 64, 40), (BF16, 128, 128), (BF16, 64, 64)])
def test_long_and_few_units(dtype, dk, dv):
    x = make(5, dtype, 1, 1, 2500, dk, dv)
    check_prefill(x, dtype)
    check_backward(x, dtype, s0=False)


@pytest.mark.parametrize("kind", ["mild", "resets", "cliff", None])
@pytest.mark.parametrize("dtype,dk,dv,T,lens", [(BF16, 128, 128, 2200, None), (BF16, 64, 64, 2048, None), (F32, 40, 64, 515, None),
                                               (BF16, 24, 56, 300, None), (BF16, 128, 128, 2700, [0, 2500, 150]),
                                               (BF16, 64, 64, 4500, [513, 0, 3900, 1]), (F32, 33, 20, 700, [10, 600, 0, 70])])
def test_walk_in_segments(kind, dtype, dk, dv, T, lens):
    """Few long units: their walk is cut into four or more segments.  Sequences shorter than one, ends inside one."""
    x = make(41, dtype, 1, 2, T, dk, dv, kind, lens)
    if lens is not None:
        for m in ("q", "k", "v", "do"):
            x[m][:, :, sum(lens):] = float("nan")
    check_prefill(x, dtype)
    check_backward(x, dtype)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,T,lens", [(2, 16, 4096, None), (1, 24, 6000, None), (1, 16, 5555, [3000, 1, 0, 700, 129, 1725])])
def test_many_chunks(d, B, H, T, lens):
    """More chunks than the device holds at once, each compared by itself with the float32 kernels on the same values,
    twice: a chunk that went wrong through its neighbour's tiles shows in one of them."""
    x = make(23, BF16, B, H, T, d, d, "mild", lens)
    y = {m: t.float() if isinstance(t, torch.Tensor) and t.dtype == BF16 else t for m, t in x.items()}
    want = [*run_prefill(y)[:1], *run_backward(y)[:4]]
    for _ in range(2):
        got = [*run_prefill(x)[:1], *run_backward(x)[:4]]
        for name, a, b in zip(("o", "dq", "dk", "dv", "dg"), got, want):
            a, b = (t.double().reshape(H * B, T, -1)[:, :T // 128 * 128].reshape(H * B, T // 128, -1) for t in (a, b))
            err = (a - b).norm(dim=-1) / b.norm(dim=-1).clamp_min(float(b.norm()) / b.shape[1] ** 0.5 / (H * B) ** 0.5 / 4)
            assert bool((err <= 2 * TOL[BF16]).all()), (name, float(err.max()), int((err > 2 * TOL[BF16]).sum()))


def test_no_decay_is_the_plain_prefill():
    x = make(3, BF16, 2, 4, 500, 128, 128, None)
    o, S = run_prefill(x)
    o2, S2 = torch.empty_like(o), x["S0"].clone()
    la.la_prefill(x["q"], x["k"], x["v"], o2, S2)
    assert ref.rel(o, ref.f64(o2)) <= 2 * TOL[BF16] and ref.rel(S, ref.f64(S2)) <= 2 * TOL_STATE


@pytest.mark.parametrize("dtype,dk,dv,T", [(F32, 32, 24, 70), (F32, 64, 64, 300)])
def test_gradient_against_differences(dtype, dk, dv, T):
    """Central differences of the library's own float32 prefill along random directions.  Its loss is a sum of some
    10^4 products, each off by at most about 2^-20 of itself: over 2 h = 0.02 that is at most about 1e-3 of the
    loss's scale, which the tolerance takes relative to |gradient| |direction|."""
    x = make(21, dtype, 1, 2, T, dk, dv)
    grads = run_backward(x)

    def loss(y):
        o, S = run_prefill(y)
        return float((o.double() * x["do"].double()).sum() + (S.double() * x["dS"].double()).sum())

    gen = torch.Generator().manual_seed(4)
    for name, d in zip(("q", "k", "v", "g", "S0"), grads):
        d = d.reshape(x[name].shape)
        u = torch.randn(x[name].shape, generator=gen).to(DEV)
        u = u / u.norm() * x[name].norm()
        h = 1e-2
        up, dn = ({**x, name: x[name] + s * h * u} for s in (1, -1))
        diff = (loss(up) - loss(dn)) / (2 * h)
        want = float((d.double() * u.double()).sum())
        assert abs(diff - want) <= 1e-3 * float(d.norm() * u.norm()) + 1e-3, name


@pytest.mark.parametrize("dtype,dk,dv", [(F32, 48, 80), (F32, 7, 9), (BF16, 64, 64), (BF16, 128, 128), (BF16, 100, 60), (F32, 128, 128)])
@pytest.mark.parametrize("B,H", [(1, 1), (3, 5), (20, 16)])
@pytest.mark.parametrize("kind", ["mild", "closed", None])
def test_decode(dtype, dk, dv, B, H, kind):
    x = make(B, dtype, B, H, 3, dk, dv, kind)
    S = x["S0"].clone()
    outs = []
    for t in range(3):
        o = torch.full((B, H, dv), float("nan"), dtype=dtype, device=DEV)
        at = [x[m][:, :, t].contiguous() if x[m] is not None else None for m in ("q", "k", "v", "g")]
        la.la_gated_decode_step(*at, o, S)
        outs.append(o)
    oo, SS = ref.prefill(x["q"], x["k"], x["v"], x["g"], x["S0"])
    assert ref.rel(torch.stack(outs, 2), oo) <= TOL[dtype] and ref.rel(S, SS) <= TOL_STATE


@pytest.mark.parametrize("dtype,dk,dv", [(F32, 128, 96), (BF16, 90, 100), (F32, 33, 50), (F32, 128, 127), (BF16, 3, 2), (F32, 1, 1)])
@pytest.mark.parametrize("units", [1, 148, 149, 296, 297, 700])
@pytest.mark.parametrize("off", [0, 1, 2])
def test_decode_sizes(dtype, dk, dv, units, off):
    """Head sizes of every divisibility, unit counts around the changes of kernel, states off 16-byte boundaries."""
    x = make(units, dtype, units, 1, 1, dk, dv)
    S = torch.empty(units * dk * dv + off, device=DEV)[off:].view(units, dk, dv)
    S.copy_(x["S0"])
    o = torch.full((units, 1, dv), float("nan"), dtype=dtype, device=DEV)
    la.la_gated_decode_step(*(x[m][:, :, 0].contiguous() for m in "qkvg"), o, S)
    oo, SS = ref.prefill(x["q"], x["k"], x["v"], x["g"], x["S0"])
    assert ref.rel(o[:, :, None], oo) <= TOL[dtype] and ref.rel(S, SS) <= TOL_STATE


@pytest.mark.parametrize("dtype,dk,dv", [(BF16, 128, 128), (F32, 48, 80), (BF16, 64, 64)])
def test_together(dtype, dk, dv):
    """As a model uses them: positions on q and k, the prompt, drafted tokens, single tokens; one long call agrees."""
    B, H, T = 2, 3, 205
    x = make(9, dtype, B, H, T, dk, dv)
    freq = torch.empty(dk // 4, device=DEV)
    la.la_rotary_init(freq, scaling="parts", factor=4.0, original=64.0)
    q, k = torch.empty_like(x["q"]), torch.empty_like(x["k"])
    la.la_rotary(x["q"], x["k"], q, k, freq, scale=1.1)
    S = x["S0"].clone()
    o = torch.full_like(x["v"], float("nan"))
    cuts = [(0, 190), (190, 198), *((t, t + 1) for t in range(198, T))]
    for a, b in cuts:
        start = torch.full((B,), a, dtype=torch.int32, device=DEV)
        part = {m: x[m][:, :, a:b].contiguous() for m in ("q", "k", "v", "g")}
        la.la_rotary(part["q"], part["k"], part["q"], part["k"], freq, start=start, scale=1.1)     # in place
        assert torch.equal(part["q"], q[:, :, a:b]) and torch.equal(part["k"], k[:, :, a:b])
        if b - a == 1:
            y = torch.empty(B, H, dv, dtype=dtype, device=DEV)
            la.la_gated_decode_step(*(part[m][:, :, 0].contiguous() for m in "qkvg"), y, S)
            o[:, :, a] = y
        else:
            y = torch.empty(B, H, b - a, dv, dtype=dtype, device=DEV)
            ws = torch.empty(la.la_gated_prefill_workspace_size(dtype, B, H, b - a, dk, dv), dtype=torch.uint8, device=DEV)
            la.la_gated_prefill(*(part[m] for m in "qkvg"), y, S, workspace=ws)
            o[:, :, a:b] = y
    oo, SS = ref.prefill(q, k, x["v"], x["g"], x["S0"])
    # the state passes three kinds of call; each adds at most its own tolerance
    assert ref.rel(o, oo) <= TOL[dtype] and ref.rel(S, SS) <= 3 * TOL_STATE
    # and the gradients of the positions are the turned back gradients
    one = make(9, dtype, B, H, T, dk, dv)
    one["q"], one["k"] = q, k
    check_backward(one, dtype)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("lens", [None, [70, 0, 190, 41]])
def test_captured_and_other_stream(lens, backward):
    """A captured graph replayed on changed inputs, and a call on a stream of its own, give what an eager call gives."""
    x = make(13, BF16, 1, 4, 301, 128, 128, "mild", lens)
    y = make(14, BF16, 1, 4, 301, 128, 128, "mild", lens)
    fn = run_backward if backward else run_prefill
    want = [t.clone() for t in fn(y)]
    live = {m: x[m].clone() for m in ("q", "k", "v", "g", "S0", "do", "dS")}
    ws = ws_for(x, backward)
    outs = {n: torch.zeros_like(live[m]) for n, m in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"), ("o", "v"))}
    st = live["S0"].clone()

    def call():
        if backward:
            st.copy_(live["dS"])
            la.la_gated_prefill_backward(live["q"], live["k"], live["v"], live["g"], live["S0"], live["do"], st, outs["dq"], outs["dk"],
                                         outs["dv"], outs["dg"], cu_seqlens=x["cu"], workspace=ws)
        else:
            st.copy_(live["S0"])
            la.la_gated_prefill(live["q"], live["k"], live["v"], live["g"], outs["o"], st, cu_seqlens=x["cu"], workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for m, t in live.items():
        t.copy_(y[m])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert la.la_device_status() == la.LA_OK
    got = [outs[n] for n in ("dq", "dk", "dv", "dg")] + [st] if backward else [outs["o"], st]
    n = 301 if lens is None else sum(lens)
    for a, b in zip(got, want):
        a, b = (t if t is st or t.shape == st.shape else t[:, :, :n] for t in (a, b))
        assert torch.equal(a, b)       # the same kernels on the same inputs: no order of execution shows


def test_two_calls_at_once():
    """Two streams, a workspace each."""
    x, y = (make(s, BF16, 2, 8, 700, 128, 128) for s in (31, 32))
    want = [[t.clone() for t in run_backward(z)] for z in (x, y)]
    ws = [ws_for(z, True) for z in (x, y)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    torch.cuda.synchronize()
    for z, w, s in zip((x, y), ws, streams):
        with torch.cuda.stream(s):
            out = [torch.empty_like(z[m]) for m in ("q", "k", "v", "g")] + [z["dS"].clone()]
            la.la_gated_prefill_backward(z["q"], z["k"], z["v"], z["g"], z["S0"], z["do"], out[4], *out[:4], workspace=w)
            got.append(out)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_prefills_at_once():
    """Three streams whose launches share the device: each one's CTAs that wait and those that they wait for start when
    others leave room.  Few units in segments, many units, packed ones."""
    xs = [make(33, BF16, 1, 3, 6000, 128, 128), make(34, BF16, 12, 16, 900, 128, 128), make(35, BF16, 1, 16, 5000, 64, 64, "mild", [4000, 0, 1000])]
    want = [[t.clone() for t in run_prefill(x)] for x in xs]
    ws = [ws_for(x, False) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        got = [(torch.empty_like(x["v"]), x["S0"].clone()) for x in xs]
        torch.cuda.synchronize()
        for x, w, s, (o, S) in zip(xs, ws, streams, got):
            with torch.cuda.stream(s):
                la.la_gated_prefill(x["q"], x["k"], x["v"], x["g"], o, S, cu_seqlens=x["cu"], workspace=w)
        torch.cuda.synchronize()
        assert la.la_device_status() == la.LA_OK
        for a, b in zip(got, want):
            assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_one_workspace_for_calls_of_many_sizes():
    """Sized for the largest call and used for each in turn, in order on one stream."""
    ws = {b: ws_for(make(1, BF16, 28, 2, 2048, 128, 128), b) for b in (False, True)}
    for B, T in ((28, 2048), (27, 2048), (1, 2048), (3, 1999), (1, 17), (28, 500)):
        x = make(B + T, BF16, B, 2, T, 128, 128)
        for fn, b in ((run_prefill, False), (run_backward, True)):
            assert all(torch.equal(s, t) for s, t in zip(fn(x, ws=ws[b]), fn(x)))


def test_more_than_2_31_elements():
    """The last head of tensors of 2^31 elements and more, against a call of its own."""
    if torch.cuda.get_device_properties(0).total_memory < 100 << 30:
        pytest.skip("needs 60 GB")
    gen = torch.Generator(device=DEV).manual_seed(6)
    B, H, T, d = 1, 130, 131072, 128
    q, k, v, do = (torch.randn(B, H, T, d, generator=gen, device=DEV, dtype=BF16).mul_(0.1) for _ in range(4))
    g = -0.1 * torch.rand(B, H, T, generator=gen, device=DEV).to(BF16)
    assert q.numel() > 1 << 31
    x = dict(q=q, k=k, v=v, g=g, do=do, S0=torch.zeros(H, d, d, device=DEV), dS=torch.zeros(H, d, d, device=DEV), cu=None, lens=None)
    y = {m: (t[:, -1:].contiguous() if t.dim() > 3 or m == "g" else t[-1:].clone()) for m, t in x.items() if t is not None}
    y.update(cu=None, lens=None)
    for fn, tail in ((run_prefill, lambda t: t[:, -1:]), (run_backward, lambda t: t[:, -1:])):
        whole = [(t[-1:] if t.shape[0] == H else tail(t)).clone() for t in fn(x)]
        torch.cuda.empty_cache()
        for a, b in zip(whole, fn(y)):        # walked whole and in segments: two sums of the same products
            assert float((a.double() - b.double()).norm() / b.double().norm()) <= (2 * TOL_STATE if a.dtype == F32 else 2.0 ** -8)


def test_without_dg_and_bad_offsets():
    x = make(17, BF16, 1, 2, 300, 64, 64, None)
    out = [torch.empty_like(x[m]) for m in ("q", "k", "v")]
    D = x["dS"].clone()
    la.la_gated_prefill_backward(x["q"], x["k"], x["v"], None, None, x["do"], D, *out, workspace=ws_for(x, True))
    full = run_backward(x, s0=False)
    assert all(torch.equal(a, b) for a, b in zip(out, full[:3])) and torch.equal(D, full[4])
    # offsets that do not rise, or leave the tensor, are empty sequences: their states stay
    y = make(18, BF16, 1, 2, 300, 64, 64, "mild", [100, 100, 100])
    y["cu"] = torch.tensor([0, 150, 40, 400], dtype=torch.int32, device=DEV)
    o, S = run_prefill(y)
    assert torch.equal(S[2:], y["S0"][2:]) and not torch.equal(S[:2], y["S0"][:2])
    assert torch.isfinite(o[:, :, :150]).all() and torch.isnan(o[:, :, 150:]).all()
    y["cu"] = torch.tensor([0, 300, 0, 300], dtype=torch.int32, device=DEV)      # the same rows twice: more chunks than there is room for
    run_prefill(y)
    run_backward(y)


def test_few_token_call_reports_a_longer_sequence():
    x = make(19, BF16, 1, 2, 40, 128, 128, "mild", [30, 10])
    o, S = torch.full_like(x["v"], float("nan")), x["S0"].clone()
    la.la_gated_prefill(x["q"], x["k"], x["v"], x["g"], o, S, cu_seqlens=x["cu"], max_seqlen=16)
    assert la.la_device_status() == la.LA_ERR_INVALID_ARG
    assert torch.equal(S[:2], x["S0"][:2]) and torch.isnan(o[:, :, :30]).all() and torch.isfinite(o[:, :, 30:]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d,rot", [(8, 8), (128, 128), (128, 96), (80, 40), (64, 2), (7, 6), (128, 0), (36, 34)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary(dtype, d, rot, interleaved):
    gen = torch.Generator().manual_seed(d + rot)
    B, H, T = 2, 3, 37
    q, k = (torch.randn(B, H, T, d, generator=gen).to(dtype).to(DEV) for _ in range(2))
    freq = torch.empty(rot // 2, device=DEV)
    la.la_rotary_init(freq)
    start = torch.tensor([0, (1 << 31) - 100], dtype=torch.int32, device=DEV)       # far: angles of 2e9
    pos = ref.f64(start)[:, None] + np.arange(T)
    for inverse, scale in ((False, 1.0), (True, 1.25)):
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        la.la_rotary(q, k, qo, ko, freq, start=start, scale=scale, interleaved=interleaved, inverse=inverse)
        for x, y in ((q, qo), (k, ko)):
            r = ref.rotary(x, pos, freq, scale, interleaved, inverse)
            # float32: the angle within 2^-22 of a turn, sine and cosine, three roundings; bf16: one rounding
            assert ref.rel(y, r) <= (2.0 ** -8 if dtype == BF16 else 2.0 ** -20)
            assert torch.equal(y[..., rot:], x[..., rot:])
    # turned forth and back: two roundings of each type
    one = torch.empty_like(q)
    la.la_rotary(q, None, one, None, freq, start=start, interleaved=interleaved)
    la.la_rotary(one, None, one, None, freq, start=start, interleaved=interleaved, inverse=True)
    assert ref.rel(one, ref.f64(q)) <= (2 * 2.0 ** -8 if dtype == BF16 else 2.0 ** -19)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d,rot", [(96, 88), (64, 36), (72, 20), (128, 50)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,H,T", [(1, 9, 5), (2, 16, 700), (8, 16, 2000)])
def test_rotary_widths(dtype, d, rot, interleaved, B, H, T):
    """Accesses of every width, few heads a thread and many, and tensors above the size from which they stream."""
    gen = torch.Generator(device=DEV).manual_seed(d + T)
    q, k = (torch.randn(B, H, T, d, generator=gen, device=DEV).to(dtype) for _ in range(2))
    freq = torch.empty(rot // 2, device=DEV)
    la.la_rotary_init(freq)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    la.la_rotary(q, k, qo, ko, freq, interleaved=interleaved)
    angle = torch.arange(T, device=DEV).double()[:, None] * freq.double()
    c, s = angle.cos(), angle.sin()
    for x, y in ((q, qo), (k, ko)):
        x, y = x.double(), y.double()
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
        want = x.clone()
        if interleaved:
            want[..., 0:rot:2], want[..., 1:rot:2] = a * c - b * s, b * c + a * s
        else:
            want[..., :rot // 2], want[..., rot // 2:rot] = a * c - b * s, b * c + a * s
        assert float((y - want).norm() / want.norm()) <= (2.0 ** -8 if dtype == BF16 else 2.0 ** -20)
        assert torch.equal(y[..., rot:], want[..., rot:])


@pytest.mark.parametrize("lens,behind", [([5, 0, 20, 1], 3), ([40], 0), ([0, 3], 0)])
def test_rotary_packed(lens, behind):
    gen = torch.Generator().manual_seed(1)
    T, d = sum(lens) + behind, 64
    q = torch.randn(1, 4, T, d, generator=gen).to(DEV)
    cu = torch.tensor([0, *np.cumsum(lens)], dtype=torch.int32, device=DEV)
    start = torch.arange(len(lens), dtype=torch.int32, device=DEV) * 1000
    freq = torch.empty(d // 2, device=DEV)
    la.la_rotary_init(freq, scaling="ntk", factor=4.0)
    out = torch.full_like(q, float("nan"))
    la.la_rotary(q, None, out, None, freq, start=start, cu_seqlens=cu)
    pos = np.concatenate([1000 * n + np.arange(m) for n, m in enumerate(lens)])[None]
    n = sum(lens)
    assert torch.isnan(out[:, :, n:]).all()
    assert ref.rel(out[:, :, :n], ref.rotary(q[:, :, :n], pos, freq, 1.0, False, False)) <= 2.0 ** -20


def test_rotary_misaligned_tensors():
    gen = torch.Generator().manual_seed(2)
    base = torch.randn(2 * 3 * 5 * 64 + 1, generator=gen).to(BF16).to(DEV)
    q = base[1:].view(2, 3, 5, 64)
    freq = torch.empty(32, device=DEV)
    la.la_rotary_init(freq)
    out = torch.empty_like(q)
    la.la_rotary(q, None, out, None, freq)
    same = torch.empty_like(out)
    la.la_rotary(q.clone(), None, same, None, freq)
    assert torch.equal(out, same)


@pytest.mark.parametrize("scaling,kw", [("plain", {}), ("linear", dict(factor=8.0)), ("ntk", dict(factor=4.0)),
                                        ("parts", dict(factor=8.0, original=8192.0)),
                                        ("parts", dict(factor=4.0, original=4096.0, beta_fast=4.0, beta_slow=1.0))])
@pytest.mark.parametrize("rot,base", [(2, 1e4), (64, 1e4), (128, 5e5)])
def test_rotary_table(scaling, kw, rot, base):
    freq = torch.empty(rot // 2, device=DEV)
    la.la_rotary_init(freq, base=base, scaling=scaling, **kw)
    i = np.arange(rot // 2)
    b = base * (kw["factor"] ** (rot / (rot - 2)) if scaling == "ntk" and rot > 2 else 1.0)
    f = b ** (-2.0 * i / rot)
    if scaling == "linear":
        f = f / kw["factor"]
    if scaling == "parts":
        fast, slow = kw.get("beta_fast", 32.0), kw.get("beta_slow", 1.0)
        keep = np.clip((kw["original"] * f / (2 * np.pi) - slow) / (fast - slow), 0, 1)
        f = f * keep + f / kw["factor"] * (1 - keep)
    assert np.allclose(ref.f64(freq), f, rtol=2.0 ** -23, atol=0)

"""The gated recurrence and rotary positions without a GPU: the float64 definitions against each other, and every
refusal that the host makes before a launch."""
import ctypes

import numpy as np
import pytest
import torch

import gated_ref as ref
import recurrent_decode_la_b200 as la
from recurrent_decode_la_b200 import build as labuild


@pytest.fixture(scope="module")
def lib():
    labuild.build()
    return la.load_library()


def _inputs(seed, U, T, dk, dv):
    r = np.random.default_rng(seed)
    n = r.standard_normal
    return (n((U, T, dk)), n((U, T, dk)), n((U, T, dv)), -np.abs(n((U, T))), n((U, dk, dv)), n((U, T, dv)), n((U, dk, dv)))


def test_reference_gradient_against_differences():
    """Central differences of the float64 forward: their error is of the order h^2 times third derivatives, and
    2^-53 / h by rounding; with h = 1e-5 both are below 1e-9 of values of order 10."""
    q, k, v, g, S0, do, dS = _inputs(1, 2, 7, 3, 4)

    def loss(*x):
        o, S = ref.forward(*x)
        return (o * do).sum() + (S[-1] * dS).sum()

    grads = ref.backward(q, k, v, g, S0, do, dS)
    args = [q, k, v, g, S0]
    r = np.random.default_rng(2)
    for i, d in enumerate(grads):
        u = r.standard_normal(args[i].shape)
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + 1e-5 * u, args[i] - 1e-5 * u
        diff = (loss(*up) - loss(*dn)) / 2e-5
        assert abs(diff - (d * u).sum()) < 1e-6 * max(1.0, abs(diff)), i


def test_reference_gate_zero_is_the_plain_recurrence():
    from oracle import la_oracle as ora
    q, k, v, g, S0, _, _ = _inputs(3, 2, 9, 3, 4)
    o, S = ref.forward(q, k, v, 0 * g, S0)
    oo, SS = ora.recurrent(q[None], k[None], v[None], S0[None])
    assert np.allclose(o, oo[0], rtol=1e-12, atol=1e-12) and np.allclose(S[-1], SS[0], rtol=1e-12, atol=1e-12)


def test_kernel_choice(lib):
    assert la.la_gated_prefill_kernel(torch.bfloat16, 8, 128, 128) == "short"
    assert la.la_gated_prefill_kernel(torch.bfloat16, 17, 128, 128) == "tc"
    assert la.la_gated_prefill_kernel(torch.bfloat16, 17, 64, 64) == "tc"
    assert la.la_gated_prefill_kernel(torch.bfloat16, 17, 128, 64) == "simt"
    assert la.la_gated_prefill_kernel(torch.float32, 17, 128, 128) == "simt"
    assert la.la_gated_prefill_kernel(torch.float32, 777, 48, 80) == "simt"
    assert la.la_gated_prefill_kernel(torch.float32, 8, 48, 80) == "simt"
    assert la.la_gated_prefill_kernel(torch.bfloat16, 8, 129, 128) == "unsupported"


@pytest.mark.parametrize("dtype,dk,dv", [(torch.bfloat16, 128, 128), (torch.bfloat16, 64, 64), (torch.float32, 128, 40)])
@pytest.mark.parametrize("size", [la.la_gated_prefill_workspace_size, la.la_gated_prefill_backward_workspace_size])
@pytest.mark.parametrize("packed", [False, True])
def test_a_workspace_fits_smaller_calls(lib, dtype, dk, dv, size, packed):
    """A program sizes its workspace for the largest call: none with fewer sequences, heads or tokens needs more."""
    Ts = [17, 128, 500, 1024, 2048, 2049, 5000, 5121, 8192, 40000]
    for n in (1, 2, 5, 8, 27, 28, 60):
        for H in (1, 3, 16):
            sizes = [size(dtype, 1, H, T, dk, dv, n) if packed else size(dtype, n, H, T, dk, dv) for T in Ts]
            assert sizes == sorted(sizes)
    for T in Ts:
        sizes = [size(dtype, 1, 1, T, dk, dv, n) if packed else size(dtype, n, 1, T, dk, dv) for n in range(1, 160)]
        assert sizes == sorted(sizes)


def test_workspace_sizes(lib):
    # a float32 state per chunk of 32 tokens and head; twice that for the gradient
    assert la.la_gated_prefill_workspace_size(torch.float32, 2, 3, 65, 64, 32) == 2 * 3 * 3 * 64 * 32 * 4
    assert la.la_gated_prefill_backward_workspace_size(torch.float32, 2, 3, 65, 64, 32) == 2 * 2 * 3 * 3 * 64 * 32 * 4
    # packed: two chunks of 64 rows and one more for each of five sequences, after six offsets
    assert la.la_gated_prefill_workspace_size(torch.float32, 1, 3, 64, 64, 32, 5) == 256 + 3 * 7 * 64 * 32 * 4
    # tensor cores: a bf16 state per chunk of 128, after the queue of chunks; without the queue twice for the gradient
    assert la.la_gated_prefill_workspace_size(torch.bfloat16, 2, 3, 129, 64, 64) == 256 + 2 * 2 * 3 * 64 * 64 * 2
    assert la.la_gated_prefill_backward_workspace_size(torch.bfloat16, 2, 3, 129, 64, 64) == 2 * 2 * 2 * 3 * 64 * 64 * 2
    # the few-token kernel needs none, unless the longest packed sequence is not known
    assert la.la_gated_prefill_workspace_size(torch.bfloat16, 4, 4, 16, 128, 128) == 0
    assert la.la_gated_prefill_workspace_size(torch.bfloat16, 1, 4, 16, 128, 128, 2) > 0
    for bad in ((0, 3, 65), (2, 0, 65), (2, 3, 0), (2, -3, 65)):
        assert la.la_gated_prefill_workspace_size(torch.float32, *bad, 64, 32) == 0


def _prefill(lib, **kw):
    a = dict(q=16, k=16, v=16, g=16, o=16, state=16, dtype=0, B=1, H=1, T=40, dk=8, dv=8, cu=None, n=0, most=0, ws=None, wsb=0)
    a.update(kw)
    return lib.la_gated_prefill(*a.values(), None)


def _backward(lib, **kw):
    a = dict(q=16, k=16, v=16, g=16, s0=16, do=16, ds=16, dq=16, dk_=16, dv_=16, dg=16, dtype=0, B=1, H=1, T=40, dk=8, dv=8,
             cu=None, n=0, ws=None, wsb=0)
    a.update(kw)
    return lib.la_gated_prefill_backward(*a.values(), None)


@pytest.mark.parametrize("call", [_prefill, _backward])
def test_sequence_refusals(lib, call):
    inv, uns = la.LA_ERR_INVALID_ARG, la.LA_ERR_UNSUPPORTED
    assert call(lib, dtype=7) == inv
    for bad in ({"B": -1}, {"H": -1}, {"T": -1}, {"dk": 0}, {"dv": -4}):
        assert call(lib, **bad) == inv
    assert call(lib, B=2, cu=16, n=1) == inv          # packed needs B == 1
    assert call(lib, cu=16, n=-1) == inv
    assert call(lib, dk=129) == uns and call(lib, dv=200) == uns and call(lib, T=1 << 31) == uns
    for name in ("q", "k", "v"):
        assert call(lib, **{name: None}) == inv
    assert call(lib) == inv                            # no workspace
    assert b"workspace of" in lib.la_last_cuda_error()
    assert call(lib, ws=16, wsb=64) == inv             # too small
    assert call(lib, ws=8, wsb=1 << 20) == inv         # misaligned
    # nothing to do, even with NULL pointers
    for empty in ({"B": 0}, {"H": 0}, {"T": 0}, {"cu": 16, "n": 0}):
        assert call(lib, q=None, k=None, v=None, g=None, **empty) == la.LA_OK


def test_more_refusals(lib):
    inv, uns = la.LA_ERR_INVALID_ARG, la.LA_ERR_UNSUPPORTED
    assert _prefill(lib, o=None) == inv and _prefill(lib, state=None) == inv
    assert _prefill(lib, dtype=1, T=8, dk=64, dv=64, state=8) == uns      # few tokens, state not 16-byte aligned
    for name in ("q", "k", "v", "o", "state"):                            # tensor cores: all of them
        assert _prefill(lib, dtype=1, T=80, dk=64, dv=64, ws=256, wsb=1 << 20, **{name: 8}) == uns, name
    for name in ("q", "k", "v", "s0", "do", "ds", "dq", "dk_", "dv_"):
        assert _backward(lib, dtype=1, T=80, dk=64, dv=64, ws=256, wsb=1 << 20, **{name: 8}) == uns, name
    for name in ("do", "ds", "dq", "dk_", "dv_"):
        assert _backward(lib, **{name: None}) == inv

    def decode(**kw):
        a = dict(q=16, k=16, v=16, g=16, o=16, state=16, dtype=0, B=1, H=1, dk=8, dv=8)
        a.update(kw)
        return lib.la_gated_decode_step(*a.values(), None)

    assert decode(dtype=3) == inv and decode(B=-1) == inv and decode(dk=0) == inv and decode(dv=129) == uns
    assert decode(q=None) == inv and decode(state=None) == inv and decode(B=0, q=None) == la.LA_OK

    def init(**kw):
        a = dict(freq=16, rot=8, base=1e4, scaling=0, factor=1.0, original=0.0, fast=32.0, slow=1.0)
        a.update(kw)
        return lib.la_rotary_init(*a.values(), None)

    for bad in ({"rot": 3}, {"rot": -2}, {"base": 0.0}, {"base": float("nan")}, {"scaling": 4}, {"scaling": -1}, {"scaling": 1, "factor": 0.0},
                {"scaling": 3, "factor": 2.0}, {"scaling": 3, "factor": 2.0, "original": 1e3, "fast": 1.0}, {"freq": None}):
        assert init(**bad) == inv, bad
    assert init(rot=0, freq=None) == la.LA_OK

    def rotary(**kw):
        a = dict(q=16, k=16, qo=16, ko=16, dtype=0, B=1, H=1, T=4, d=8, rot=8, freq=16, start=None, scale=1.0, il=0, inv=0, cu=None, n=0)
        a.update(kw)
        return lib.la_rotary(*a.values(), None)

    for bad in ({"dtype": 2}, {"B": -1}, {"H": -1}, {"T": -1}, {"d": 0}, {"rot": 7}, {"rot": -2}, {"rot": 10}, {"B": 2, "cu": 16, "n": 1},
                {"cu": 16, "n": -1}, {"q": None}, {"qo": None}, {"k": None}, {"ko": None}, {"freq": None}):
        assert rotary(**bad) == inv, bad
    assert rotary(d=256, rot=8) == uns and rotary(T=1 << 31) == uns
    for empty in ({"B": 0}, {"H": 0}, {"T": 0}, {"cu": 16, "n": 0}):
        assert rotary(q=None, **empty) == la.LA_OK


def test_binding_refusals():
    """The binding checks shapes, types and devices before it touches the library."""
    z = torch.zeros
    q, v, g, S = z(2, 3, 5, 8), z(2, 3, 5, 4), z(2, 3, 5), z(6, 8, 4)
    ok = (q, q, v, g, v, S)

    def bad(fn, *args, **kw):
        with pytest.raises(ValueError):
            fn(*args, **kw)

    p = la.la_gated_prefill
    bad(p, *ok)                                             # tensors of the CPU
    bad(p, q.double(), q, v, g, v, S)
    bad(p, q, q[:, :, :4], v, g, v, S)
    bad(p, q, q, v[:, :2], g, v, S)
    bad(p, q, q, v, g[:1], v, S)
    bad(p, q, q, v, g, v[..., :3], S)
    bad(p, q, q, v, g, v, S[:5])
    bad(p, q, q, v, g, v, S, cu_seqlens=torch.tensor([0, 5], dtype=torch.int32))
    bad(p, q, q, v, g, v, S, cu_seqlens=torch.tensor([0, 5]))
    bad(p, q[0], q[0], v[0], g[0], v[0], S)
    b = la.la_gated_prefill_backward
    good = dict(q=q, k=q, v=v, g=g, state0=S, do=v, dstate=S, dq=q, dk=q, dv=v, dg=g)
    for name, x in (("do", q), ("dq", v), ("dk", v), ("dv", q), ("dg", q), ("state0", S[:2]), ("dstate", S[:2])):
        bad(b, **{**good, name: x})
    t = la.la_gated_decode_step
    bad(t, q[:, :, 0], q[:, :, 0], v[:, :, 0], g[:, :, 0], v[:, :, 0], S)
    bad(t, q[:, :, 0], q[:, :, 0], v[:, :, 0], g, v[:, :, 0], S)
    bad(t, q[:, :, 0], q[:, :, 0], v[:, :, 0], g[:, :, 0], v[:, :, 0], S[:3])
    r = la.la_rotary
    f = z(4)
    bad(r, q, q, q, q, f)
    bad(r, q, None, q, q, f)
    bad(r, q, v, q, v, f)
    bad(r, q, q, q, q, z(5))
    bad(r, q, q, q, q, f, start=z(2))
    bad(r, q, q, q, q, f, start=z(3, dtype=torch.int32))
    bad(la.la_rotary_init, f, scaling="other")
    bad(la.la_rotary_init, z(2, 2))


def test_binding_argument_checks():
    """Each property that the ordinary call's one test covers is refused by itself."""
    from recurrent_decode_la_b200 import binding

    class Fake:
        dtype, shape, device, is_cuda, dev, contiguous = torch.float32, torch.Size((2, 3)), "cuda:1", True, 1, True

        def __init__(self, **kw):
            self.__dict__.update(kw)

        def get_device(self):
            return self.dev

        def is_contiguous(self):
            return self.contiguous

        def data_ptr(self):
            return 4096

        def numel(self):
            return 6

    def check(t):
        return binding._arg(t, "x", (2, 3), torch.float32, 1)

    assert check(Fake()) == 4096
    for bad in (dict(dtype=torch.bfloat16), dict(shape=torch.Size((3, 2))), dict(dev=0), dict(dev=-1, is_cuda=False), dict(contiguous=False)):
        with pytest.raises(ValueError):
            check(Fake(**bad))
    with pytest.raises(ValueError):
        binding._floats(Fake(), "x", 7, 1)

"""The gated recurrence, its gradient and rotary positions in float64, from their definitions, token by token.

Units are [U, T, d] numpy arrays; ``units`` / ``rows`` convert the library's dense and packed layouts."""
from __future__ import annotations

import numpy as np


def f64(x) -> np.ndarray:
    return x.detach().double().cpu().numpy() if hasattr(x, "detach") else np.asarray(x, np.float64)


def forward(q, k, v, g, S0):
    """S_t = e^{g_t} S_{t-1} + k_t v_t^T, o_t = q_t^T S_t; returns o and every state S_0 .. S_T."""
    S, o, states = S0.copy(), np.zeros_like(v), [S0.copy()]
    a = np.exp(g)
    for t in range(q.shape[1]):
        S = a[:, t, None, None] * S + k[:, t, :, None] * v[:, t, None, :]
        o[:, t] = np.einsum("ud,udn->un", q[:, t], S)
        states.append(S)
    return o, states


def backward(q, k, v, g, S0, do, dS):
    _, S = forward(q, k, v, g, S0)
    a = np.exp(g)
    dq, dk, dv, dg, D = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v), np.zeros_like(g), dS.copy()
    for t in reversed(range(q.shape[1])):
        D = D + q[:, t, :, None] * do[:, t, None, :]
        dq[:, t] = np.einsum("udn,un->ud", S[t + 1], do[:, t])
        dk[:, t] = np.einsum("udn,un->ud", D, v[:, t])
        dv[:, t] = np.einsum("ud,udn->un", k[:, t], D)
        D = a[:, t, None, None] * D
        dg[:, t] = (D * S[t]).sum((1, 2))
    return dq, dk, dv, dg, D


def split(x, lens):
    """The sequences of [B,H,T,..]: dense (lens None) one list entry [B*H,T,..]; packed one [H,len,..] each."""
    x = f64(x)
    if lens is None:
        return [x.reshape(-1, *x.shape[2:])]
    ends = np.concatenate([[0], np.cumsum(lens)])
    return [x[0][:, a:b] for a, b in zip(ends, ends[1:])]


def join(parts, like, lens):
    if lens is None:
        return parts[0].reshape(like.shape)
    out = np.full(like.shape, np.nan)
    at = 0
    for y, n in zip(parts, lens):
        out[0][:, at:at + n] = y
        at += n
    return out


def states_of(S, lens, H):
    S = f64(S).reshape(-1, *S.shape[-2:])
    return [S] if lens is None else [S[n * H:(n + 1) * H] for n in range(len(lens))]


def prefill(q, k, v, g, S0, lens=None):
    g0 = np.zeros(q.shape[:3]) if g is None else g
    o, S = [], []
    for x in zip(*(split(t, lens) for t in (q, k, v, g0)), states_of(S0, lens, q.shape[1])):
        oo, ss = forward(*x)
        o.append(oo)
        S.append(ss[-1])
    return join(o, v, lens), np.concatenate(S)


def prefill_backward(q, k, v, g, S0, do, dS, lens=None):
    g0 = np.zeros(q.shape[:3]) if g is None else g
    H = q.shape[1]
    got = [backward(*x) for x in zip(*(split(t, lens) for t in (q, k, v, g0)), states_of(S0, lens, H), split(do, lens),
                                     states_of(dS, lens, H))]
    like = (q, k, v, g0)
    return [join([x[i] for x in got], like[i], lens) for i in range(4)] + [np.concatenate([x[4] for x in got])]


def rotary(x, pos, freq, scale, interleaved, inverse):
    """x [B,H,T,d], pos [B or 1,T]."""
    x = f64(x)
    f = f64(freq)
    rot = 2 * f.size
    angle = np.asarray(pos, np.float64)[:, None, :, None] * f
    turn = scale * np.exp(-1j * angle if inverse else 1j * angle)
    y = x.copy()
    ia = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    z = (x[..., ia] + 1j * x[..., ib]) * turn
    y[..., ia], y[..., ib] = z.real, z.imag
    return y


def rel(x, ref) -> float:
    """2-norm of the difference over 2-norm of the reference (of finite values; a non-finite one is an error)."""
    x, ref = f64(x).ravel(), np.asarray(ref, np.float64).ravel()
    if not np.isfinite(x).all():
        return float("inf")
    n = np.linalg.norm(ref)
    d = np.linalg.norm(x - ref)
    return float(d / n) if n else float(d)

"""Cases, plain forms and float64 definitions of the gated recurrence and of rotary positions.

Four operators:

* ``prefill``   S_t = exp(g_t) S_{t-1} + k_t v_t^T,  o_t = q_t^T S_t   over whole sequences, dense or packed;
* ``backward``  the gradients of q, k, v, g and of the incoming state, given those of o and of the final state;
* ``decode``    one token of the recurrence for every (sequence, head), the state updated in place;
* ``rotary``    q and k turned by their positions (pairs in halves or interleaved, part of the head, scaled tables).

``run`` with ``own`` false computes the plain form: the chunk form with batched products in float32 (positions'
angles and sums of log gates in float64), its gradients by differentiating that form.  With ``own`` true it makes the
calls a user makes.  ``exact`` follows the definitions token by token in float64.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # a whole training or scoring batch: the shape the framework's own benchmark runs
        {"name": "prefill_b8h16_t8192_d128", "op": "prefill", "dtype": "bf16", "B": 8, "H": 16, "T": 8192, "dk": 128, "dv": 128, "seqs": 0},
        # a serving batch of prompts of very different lengths, packed
        {"name": "prefill_packed24_h16_t30011", "op": "prefill", "dtype": "bf16", "B": 1, "H": 16, "T": 30011, "dk": 128, "dv": 128, "seqs": 24},
        # drafted tokens taken from a saved state: eight per sequence
        {"name": "prefill_b16h16_t8_d128", "op": "prefill", "dtype": "bf16", "B": 16, "H": 16, "T": 8, "dk": 128, "dv": 128, "seqs": 0},
        # a float32 model with heads that are no power of two and an odd length
        {"name": "prefill_f32_b2h6_t777", "op": "prefill", "dtype": "f32", "B": 2, "H": 6, "T": 777, "dk": 48, "dv": 80, "seqs": 0},
        # a training step of a small model: few heads, medium length
        {"name": "backward_b4h8_t2048_d64", "op": "backward", "dtype": "bf16", "B": 4, "H": 8, "T": 2048, "dk": 64, "dv": 64, "seqs": 0},
        # a training step at the benchmark's width
        {"name": "backward_b4h16_t8192_d128", "op": "backward", "dtype": "bf16", "B": 4, "H": 16, "T": 8192, "dk": 128, "dv": 128, "seqs": 0},
        # documents packed into one row of a training batch, ragged
        {"name": "backward_packed9_h8_t8191", "op": "backward", "dtype": "bf16", "B": 1, "H": 8, "T": 8191, "dk": 128, "dv": 128, "seqs": 9},
        # the same in float32 at odd sizes
        {"name": "backward_f32_b2h3_t515", "op": "backward", "dtype": "f32", "B": 2, "H": 3, "T": 515, "dk": 64, "dv": 40, "seqs": 0},
        # one token for a small batch: latency
        {"name": "decode_b8h16_d128", "op": "decode", "dtype": "bf16", "B": 8, "H": 16, "T": 1, "dk": 128, "dv": 128, "seqs": 0},
        # one token for a large serving batch: the states do not fit the caches
        {"name": "decode_b256h32_d128", "op": "decode", "dtype": "bf16", "B": 256, "H": 32, "T": 1, "dk": 128, "dv": 128, "seqs": 0},
        # q and k of a whole batch, half layout, all of the head
        {"name": "rotary_b8h16_t8192_d128", "op": "rotary", "dtype": "bf16", "B": 8, "H": 16, "T": 8192, "dk": 128, "dv": 128, "seqs": 0,
         "rot": 128, "layout": "half", "scaling": "none", "far": 0, "inverse": False},
        # q and k of one token for every sequence, far positions under a scaled table, a quarter of the head left alone
        {"name": "rotary_b64h32_t1_far", "op": "rotary", "dtype": "bf16", "B": 64, "H": 32, "T": 1, "dk": 128, "dv": 128, "seqs": 0,
         "rot": 96, "layout": "interleaved", "scaling": "yarn", "far": 1 << 20, "inverse": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "backward", "backward", "decode", "rotary"])
    dtype = "bf16" if rng.random() < 0.7 else "f32"
    if op == "rotary":
        d = rng.choice([32, 64, 80, 96, 128])
        rot = 2 * rng.randint(1, d // 2) if rng.random() < 0.5 else d
        B, H = _log_int(rng, 1, 64), _log_int(rng, 1, 32)
        T = _log_int(rng, 1, 16384)
        while B * H * T * d * (2 if dtype == "f32" else 1) > 8 * 16 * 8192 * 128:
            B, T = max(1, B // 2), max(1, T * 2 // 3)
        seqs = rng.randint(1, 12) if rng.random() < 0.3 and T >= 16 else 0
        return {"op": op, "dtype": dtype, "B": 1 if seqs else B, "H": H, "T": T, "dk": d, "dv": d, "seqs": seqs, "rot": rot,
                "layout": rng.choice(["half", "interleaved"]), "scaling": rng.choice(["none", "linear", "ntk", "yarn"]),
                "far": rng.choice([0, 0, 5000, 1 << 20]), "inverse": rng.random() < 0.4}
    if dtype == "bf16" and rng.random() < 0.75:
        dk = dv = rng.choice([64, 128])
    else:
        dk, dv = rng.randint(8, 128), rng.randint(8, 128)
    B, H = _log_int(rng, 1, 16), _log_int(rng, 1, 32)
    if op == "decode":
        B = _log_int(rng, 1, 256)
        return {"op": op, "dtype": dtype, "B": B, "H": H, "T": 1, "dk": dk, "dv": dv, "seqs": 0}
    T = _log_int(rng, 1, 32768)
    most = (1 << 20 if op == "prefill" else 1 << 19) if dtype == "bf16" and dk == dv and dk in (64, 128) else 1 << 15
    while B * H * T > most:
        B, H, T = max(1, B * 2 // 3), max(1, H * 3 // 4), max(1, T * 3 // 4)
    seqs = rng.randint(1, 16) if rng.random() < 0.35 and T >= 32 else 0
    return {"op": op, "dtype": dtype, "B": 1 if seqs else B, "H": H, "T": T, "dk": dk, "dv": dv, "seqs": seqs}


def _lengths(case):
    """The packed sequences' lengths: random cuts of T, so short, empty and long ones occur together."""
    rng = random.Random("%(T)d %(H)d %(seqs)d" % case)
    cuts = sorted(rng.randint(0, case["T"]) for _ in range(case["seqs"] - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [case["T"]])]


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    units, T, dk, dv = case["B"] * case["H"], case["T"], case["dk"], case["dv"]
    rows, states = units * T, (case["seqs"] or case["B"]) * case["H"]
    if case["op"] == "rotary":
        return {"bytes": 4 * rows * dk * es, "flops": 6 * rows * case["rot"]}
    if case["op"] == "backward":  # q k v g do in, dq dk dv dg out; S_0 and dS_T in, dS_0 out
        return {"bytes": rows * (4 * dk + 3 * dv + 2) * es + 3 * states * dk * dv * 4, "flops": 10 * rows * dk * dv}
    return {"bytes": rows * (2 * dk + 2 * dv + 1) * es + 2 * states * dk * dv * 4, "flops": 4 * rows * dk * dv}


# ----------------------------------------------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------------------------------------------
def _table(case):
    """Angular frequencies of the pairs, float32: a base of 10000, stretched eightfold where the case says so."""
    rot, base, factor, orig = case["rot"], 10000.0, 8.0, 8192.0
    i = torch.arange(rot // 2, dtype=torch.float64)
    kind = case["scaling"]
    if kind == "ntk" and rot > 2:
        base *= factor ** (rot / (rot - 2))
    f = base ** (-2 * i / rot)
    if kind == "linear":
        f = f / factor
    elif kind == "yarn":  # pairs that turn often keep their frequency, slow ones are stretched, a ramp between
        turns = orig * f / (2 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1 - keep)
    return f.float(), (0.1 * math.log(factor) + 1.0 if kind == "yarn" else 1.0)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dt = _TYPES[case["dtype"]]
    B, H, T, dk, dv = case["B"], case["H"], case["T"], case["dk"], case["dv"]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    s = {"case": case}
    if case["seqs"]:
        lens = _lengths(case)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s["lens"], s["cu"] = lens, torch.tensor(cu, dtype=torch.int32, device=dev)
    if case["op"] == "rotary":
        s["q"], s["k"] = randn(B, H, T, dk).to(dt), randn(B, H, T, dk).to(dt)
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        n = case["seqs"] or B
        s["start"] = torch.randint(0, case["far"] + 1, (n,), generator=gen, device=dev, dtype=torch.int32)
        f, s["scale"] = _table(case)
        s["freq"] = f.to(dev)
        return s
    tok = (B, H) if case["op"] == "decode" else (B, H, T)
    # keys of unit length, queries and values of ordinary size, gates as a sigmoid of a projection gives them: memories
    # of a few to a few hundred tokens
    s["q"] = (randn(*tok, dk) / math.sqrt(dk)).to(dt)
    k = randn(*tok, dk)
    s["k"] = (k / k.norm(dim=-1, keepdim=True)).to(dt)
    s["v"] = randn(*tok, dv).to(dt)
    s["g"] = torch.nn.functional.logsigmoid(randn(*tok) * 1.2 + 3.5).to(dt)
    n = (case["seqs"] or B) * H
    s["state"] = randn(n, dk, dv) * 0.3
    if case["op"] == "backward":
        s["do"] = randn(*tok, dv).to(dt)
        s["dstate"] = randn(n, dk, dv) * 0.3
        for name, like in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g")):
            s[name] = torch.empty_like(s[like])
    else:
        s["o"] = torch.empty_like(s["v"])
    return s


# ----------------------------------------------------------------------------------------------------------------
# Rows of the packed layout as padded units, and back
# ----------------------------------------------------------------------------------------------------------------
def _pad_rows(s):
    """For packed input: the row of every (sequence, place), and whether it is one."""
    lens = torch.tensor(s["lens"], device=s["cu"].device)
    place = torch.arange(max(s["lens"]), device=lens.device)
    there = place[None] < lens[:, None]
    return torch.where(there, s["cu"][:-1, None].long() + place[None], 0), there


def _units(s, x, feat):
    """[B,H,T,(d)] as [units, rows, (d)]; packed rows go to their own units, padded with zeros."""
    if not s["case"]["seqs"]:
        return x.reshape(-1, *x.shape[2:])
    row, there = _pad_rows(s)
    y = x[0][:, row].transpose(0, 1)  # [N,H,L,(d)]
    m = there[:, None, :, None] if feat else there[:, None, :]
    return (y * m.to(y.dtype)).reshape(-1, *y.shape[2:])


def _rows(s, y, like):
    """The inverse of _units."""
    if not s["case"]["seqs"]:
        return y.reshape(like.shape)
    row, there = _pad_rows(s)
    N, H = there.shape[0], s["case"]["H"]
    y = y.reshape(N, H, *y.shape[1:]).transpose(0, 1)
    out = torch.zeros(like.shape, dtype=y.dtype, device=y.device)
    out[0][:, row[there]] = y[:, there]
    return out


# ----------------------------------------------------------------------------------------------------------------
# The plain form
# ----------------------------------------------------------------------------------------------------------------
def _chunk_form(q, k, v, g, s0):
    """q, k [U,T,dk], v [U,T,dv], g [U,T] and s0 [U,dk,dv], float32: o and the final state."""
    U, T, dk = q.shape
    dv = v.shape[-1]
    C = 64
    while C * C < 2 * T:
        C *= 2
    n = -(-T // C)
    pad = n * C - T
    pad2 = torch.nn.functional.pad
    q, k, v = (pad2(x, (0, 0, 0, pad)).reshape(U, n, C, -1) for x in (q, k, v))
    G = pad2(g, (0, pad)).double().reshape(U, n, C).cumsum(-1)
    low = torch.ones(C, C, dtype=torch.bool, device=q.device).tril()
    decay = torch.where(low, G[..., :, None] - G[..., None, :], -math.inf).float().exp()
    o = ((q @ k.transpose(-1, -2)) * decay) @ v
    add = (k * (G[..., -1:] - G).float().exp()[..., None]).transpose(-1, -2) @ v  # [U,n,dk,dv]
    # the state before chunk c is the sum over the chunks before it (and s0) of what they add, decayed
    L = torch.cat([torch.zeros_like(G[:, :1, 0]), G[..., -1].cumsum(1)], 1)  # [U,n+1]
    add = torch.cat([s0.reshape(U, 1, dk, dv), add], 1).reshape(U, n + 1, dk * dv)
    lowc = torch.ones(n + 1, n + 1, dtype=torch.bool, device=q.device).tril()
    across = torch.where(lowc, L[:, :, None] - L[:, None, :], -math.inf).float().exp()
    states = (across @ add).reshape(U, n + 1, dk, dv)
    o = o + (q @ states[:, :-1]) * G.float().exp()[..., None]
    return o.reshape(U, n * C, dv)[:, :T], states[:, -1]


def _rotary_positions(s):
    """[B or 1, T] positions (int64)."""
    T = s["case"]["T"]
    t = torch.arange(T, device=s["q"].device)
    if not s["case"]["seqs"]:
        return s["start"].long()[:, None] + t[None]
    n = torch.repeat_interleave(torch.arange(len(s["lens"]), device=t.device), torch.tensor(s["lens"], device=t.device), output_size=T)
    return (s["start"].long()[n] + t - s["cu"].long()[n])[None]


def _rotate(s, x, wide):
    """x [B,H,T,d] turned, computed in the type `wide`."""
    case = s["case"]
    rot = case["rot"]
    angle = _rotary_positions(s).double()[:, None, :, None] * s["freq"].double()
    c = (angle.cos() * s["scale"]).to(wide)
    sn = (angle.sin() * (-s["scale"] if case["inverse"] else s["scale"])).to(wide)
    x = x.to(wide)
    if case["layout"] == "half":
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        turned = torch.cat([a * c - b * sn, b * c + a * sn], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain(s):
    op, dt = s["case"]["op"], s["q"].dtype
    f = torch.float32
    if op == "rotary":
        return {"q": _rotate(s, s["q"], f).to(dt), "k": _rotate(s, s["k"], f).to(dt)}
    if op == "decode":
        B, H, dk, dv = s["case"]["B"], s["case"]["H"], s["case"]["dk"], s["case"]["dv"]
        S = s["state"].reshape(B, H, dk, dv) * s["g"].float().exp()[..., None, None]
        S = S + s["k"].float()[..., None] * s["v"].float()[..., None, :]
        o = (s["q"].float()[..., None, :] @ S)[..., 0, :]
        s["state"].copy_(S.reshape(s["state"].shape))
        return {"o": o.to(dt), "state": s["state"]}
    q, k, v = (_units(s, s[n].float(), True) for n in ("q", "k", "v"))
    g = _units(s, s["g"].float(), False)
    if op == "prefill":
        o, S = _chunk_form(q, k, v, g, s["state"])
        s["state"].copy_(S)
        return {"o": _rows(s, o, s["v"]).to(dt), "state": s["state"]}
    leaves = [x.detach().requires_grad_() for x in (q, k, v, g, s["state"])]
    with torch.enable_grad():
        o, S = _chunk_form(*leaves)
    grads = torch.autograd.grad((o, S), leaves, (_units(s, s["do"].float(), True), s["dstate"]))
    s["dstate"].copy_(grads[4])
    out = {"d" + n: _rows(s, d, s[n]).to(dt) for n, d in zip("qkvg", grads)}
    return {**out, "dstate": s["dstate"]}


# ----------------------------------------------------------------------------------------------------------------
# The framework's calls
# ----------------------------------------------------------------------------------------------------------------
def _calls(s):
    import recurrent_decode_la_b200 as la

    case, dt = s["case"], s["q"].dtype
    B, H, T, dk, dv = case["B"], case["H"], case["T"], case["dk"], case["dv"]
    packed = {"cu_seqlens": s["cu"]} if case["seqs"] else {}
    if case["op"] == "rotary":
        la.la_rotary(s["q"], s["k"], s["q_out"], s["k_out"], s["freq"], start=s["start"], scale=s["scale"],
                     interleaved=case["layout"] == "interleaved", inverse=case["inverse"], **packed)
        return {"q": s["q_out"], "k": s["k_out"]}
    if case["op"] == "decode":
        la.la_gated_decode_step(s["q"], s["k"], s["v"], s["g"], s["o"], s["state"])
        return {"o": s["o"], "state": s["state"]}
    if packed:
        packed["max_seqlen"] = max(s["lens"])
    if "workspace" not in s:  # kept by the program from step to step
        size = la.la_gated_prefill_workspace_size if case["op"] == "prefill" else la.la_gated_prefill_backward_workspace_size
        s["workspace"] = torch.empty(size(dt, B, H, T, dk, dv, case["seqs"]), dtype=torch.uint8, device=s["q"].device)
    if case["op"] == "prefill":
        la.la_gated_prefill(s["q"], s["k"], s["v"], s["g"], s["o"], s["state"], workspace=s["workspace"], **packed)
        return {"o": s["o"], "state": s["state"]}
    la.la_gated_prefill_backward(s["q"], s["k"], s["v"], s["g"], s["state"], s["do"], s["dstate"], s["dq"], s["dk"], s["dv"], s["dg"],
                                 workspace=s["workspace"], **packed)
    return {n: s[n] for n in ("dq", "dk", "dv", "dg", "dstate")}


def run(state):
    return _calls(state) if own else _plain(state)


# ----------------------------------------------------------------------------------------------------------------
# The definitions in float64
# ----------------------------------------------------------------------------------------------------------------
def _forward64(q, k, v, a, S):
    """The recurrence token by token; S is changed in place."""
    o = torch.empty_like(v)
    for t in range(q.shape[1]):
        S.mul_(a[:, t, None, None]).baddbmm_(k[:, t, :, None], v[:, t, None, :])
        o[:, t] = torch.bmm(q[:, t, None, :], S)[:, 0]
    return o


def _backward64(q, k, v, a, S0, do, D):
    """dq_t = S_t do_t;  D_t = q_t do_t^T + a_{t+1} D_{t+1};  dk_t = D_t v_t;  dv_t = D_t^T k_t;
    dg_t = a_t <D_t, S_{t-1}>;  dS_0 = a_1 D_1.  The states are kept every `step` tokens and made again between."""
    U, T, dk = q.shape
    step = max(1, min(64, (1 << 31) // (8 * U * dk * v.shape[-1])))
    dq, dk_, dv, dg = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(a)
    S, kept = S0.clone(), []
    for t in range(T):
        if t % step == 0:
            kept.append(S.clone())
        S.mul_(a[:, t, None, None]).baddbmm_(k[:, t, :, None], v[:, t, None, :])
        dq[:, t] = torch.bmm(S, do[:, t, :, None])[..., 0]
    for c in reversed(range(len(kept))):
        t0, t1 = c * step, min(T, (c + 1) * step)
        before = [kept.pop()]
        for t in range(t0, t1 - 1):
            before.append(torch.baddbmm(before[-1] * a[:, t, None, None], k[:, t, :, None], v[:, t, None, :]))
        for t in reversed(range(t0, t1)):
            D.baddbmm_(q[:, t, :, None], do[:, t, None, :])
            dk_[:, t] = torch.bmm(D, v[:, t, :, None])[..., 0]
            dv[:, t] = torch.bmm(k[:, t, None, :], D)[:, 0]
            D.mul_(a[:, t, None, None])
            dg[:, t] = (D * before[t - t0]).sum((1, 2))
    return dq, dk_, dv, dg, D


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return {"q": _rotate64(s, s["q"]), "k": _rotate64(s, s["k"])}
    if case["op"] == "decode":
        x = {n: s[n].double().reshape(-1, 1, *s[n].shape[2:]) for n in "qkvg"}
        S = s["state"].double()
        o = _forward64(x["q"], x["k"], x["v"], x["g"].exp(), S)
        return {"o": o.reshape(s["v"].shape), "state": S}
    if not case["seqs"]:
        parts, where = [(slice(None), slice(None), slice(0, case["B"] * case["H"]))], None
    else:
        ends = s["cu"].tolist()
        H = case["H"]
        parts = [(slice(None), slice(a, b), slice(n * H, (n + 1) * H)) for n, (a, b) in enumerate(zip(ends, ends[1:]))]
    out = {}

    def put(name, like, part, x):
        if name not in out:
            out[name] = torch.zeros(like.shape, dtype=torch.float64, device=like.device)
        dest = out[name] if like.dim() == 3 and name in ("state", "dstate") else out[name][:, part[0], part[1]]
        if name in ("state", "dstate"):
            out[name][part[2]] = x
        else:
            dest.copy_(x.reshape(dest.shape))

    for part in parts:
        x = {n: s[n][:, part[0], part[1]].double() for n in ("q", "k", "v", "g")}
        x = {n: t.reshape(-1, *t.shape[2:]) for n, t in x.items()}
        S0 = s["state"][part[2]].double()
        if case["op"] == "prefill":
            S = S0.clone()
            o = _forward64(x["q"], x["k"], x["v"], x["g"].exp(), S)
            put("o", s["v"], part, o)
            put("state", s["state"], part, S)
        else:
            do = s["do"][:, part[0], part[1]].double()
            got = _backward64(x["q"], x["k"], x["v"], x["g"].exp(), S0, do.reshape(-1, *do.shape[2:]), s["dstate"][part[2]].double())
            for name, like, y in zip(("dq", "dk", "dv", "dg", "dstate"), ("q", "k", "v", "g", "dstate"), got):
                put(name, s[like], part, y)
    return out


def _rotate64(s, x):
    """Each pair as a complex number times scale * e^(i angle)."""
    case, x = s["case"], x.double()
    rot = case["rot"]
    if case["seqs"]:
        pos = torch.cat([st + torch.arange(n, dtype=torch.float64) for st, n in zip(s["start"].tolist(), s["lens"])])[None]
    else:
        pos = s["start"].cpu().double()[:, None] + torch.arange(case["T"], dtype=torch.float64)[None]
    angle = pos.to(x.device)[:, None, :, None] * s["freq"].double()
    turn = torch.polar(torch.full_like(angle, s["scale"]), -angle if case["inverse"] else angle)
    y = x.clone()
    if case["layout"] == "half":
        z = torch.complex(x[..., : rot // 2].contiguous(), x[..., rot // 2: rot].contiguous()) * turn
        y[..., : rot // 2], y[..., rot // 2: rot] = z.real, z.imag
    else:
        z = torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous()) * turn
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    return y

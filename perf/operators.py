"""The training and position operators beside the R-SWA attention, in plain form.

Two operators, each with the cases it is measured on:

* ``backward``: the gradient of the teacher-forced R-SWA attention of one
  sequence or of a pack of documents.  Per head, with P = exp(S - lse) on the
  visible (query, key) pairs and 0 elsewhere, S = scale * Q K^T,
  delta_i = sum_c O_ic dO_ic and dS = P * (dO V^T - delta):
  dV = P^T dO, dQ = scale * dS K, dK = scale * dS^T Q.
  Inputs: dO, Q, K, V [L, H, d], and what the forward left: O [L, H, d] and
  lse [H, L] (natural log of the sum of exponentials, float32).
* ``rotary``: rotary positions on queries and keys.  Pair i of a head turns by
  the angle position * theta_i (the pair (x_i, x_{i + r/2}) in the half layout,
  (x_2i, x_2i+1) interleaved); the head's elements from r on pass through.  The
  gradient is the turn by the opposite angle.

Visibility (0-based query row i, key row j, L_m reference rows, window n):
j <= i and (i < L_m or j < L_m or j > i - n); with a bidirectional prefix
i, j < L_m see each other too.  Documents of a pack see only themselves.
"""

from __future__ import annotations

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
PAGE, PROMPT, OUT_PER_PAGE = 256, 32, 400  # vision tokens and outputs per page, prompt tokens


# ------------------------------------------------------------------- cases

def _documents(text):
    """'288+412 33+7' -> (cu_seqlens, ref_lens): reference rows + outputs per document."""
    cu, refs = [0], []
    for part in text.split():
        ref, outs = part.split("+")
        refs.append(int(ref))
        cu.append(cu[-1] + int(ref) + int(outs))
    return cu, refs


def _pack(rng, rows):
    """A pack of `rows` rows: nine in ten documents have one page, the others 2 to 50."""
    left, parts = rows, []
    while left:
        pages = rng.randint(2, 50) if rng.random() < 0.1 else 1
        ref = min(PAGE * pages + PROMPT, left)
        outs = min(int(OUT_PER_PAGE * pages * rng.uniform(0.5, 1.5)), left - ref)
        parts.append(f"{ref}+{outs}")
        left -= ref + outs
    return " ".join(parts)


def _pairs(case):
    """Visible (query, key) pairs of one head."""
    cu, refs = _documents(case["docs"])
    total = 0
    for i, ref in enumerate(refs):
        outs, n = cu[i + 1] - cu[i] - ref, case["n"]
        total += ref * ref if case["bidir"] else ref * (ref + 1) // 2
        k = min(outs, n)
        total += outs * ref + k * (k + 1) // 2 + (outs - k) * n
    return total


def _backward(name, docs, n=128, H=10, d=128, dtype="bf16", bidir=False):
    return {"name": name, "op": "backward", "docs": docs, "n": n, "H": H, "d": d, "dtype": dtype, "bidir": bidir}


def _rotary(name, rows, H=10, Hk=10, d=128, dim=128, dtype="bf16", interleaved=False, inverse=False, fused=False,
            where="run", first=0, scaling="none", factor=1.0):
    return {"name": name, "op": "rotary", "rows": rows, "H": H, "Hk": Hk, "d": d, "dim": dim, "dtype": dtype,
            "interleaved": interleaved, "inverse": inverse, "fused": fused, "where": where, "first": first,
            "scaling": scaling, "factor": factor}


# A 32768-row training pack: one-page documents, a 5-page, a 9-page and a
# 14-page one, the last document cut where the pack ends.
PACK_32K = ("288+412 288+377 3616+5302 288+205 288+533 288+598 288+341 1312+2391 288+460 288+250 288+587 288+519 "
            "288+309 288+402 288+283 2336+3370 288+448 288+216 288+412 288+377 288+509 288+1731")


def listed():
    return [
        # the smallest gradient call: a short document of the tests, bound by latency
        _backward("backward-short", "100+200", n=16, H=2),
        # a one-page document fine-tuned by itself
        _backward("backward-page", "288+400"),
        # a ten-page document with an odd number of outputs
        _backward("backward-ten-pages", "2592+4001"),
        # the 32K teacher-forced sequence of a 50-page document: the largest
        _backward("backward-32k", "12832+19936"),
        # a 32K training pack of documents
        _backward("backward-pack-32k", PACK_32K),
        # no reference segment: the plain sliding window
        _backward("backward-window", "0+16384"),
        # 64-wide heads, a bidirectional reference, odd sizes
        _backward("backward-d64-bidir", "1283+3720 77+0", n=100, H=6, d=64, bidir=True),
        # float32 training of a small model
        _backward("backward-f32", "803+1208", H=10, dtype="f32"),
        # one decode step of one document: latency
        _rotary("rotary-step", 1, where="steps", first=12832),
        # one decode step of 64 ragged documents on a context stretched eightfold
        _rotary("rotary-step-64", 64, where="steps", first=100000, scaling="yarn", factor=8.0),
        # the 32K sequence, queries and keys read out of the fused projection
        _rotary("rotary-32k", 32768, fused=True),
        # the gradient of interleaved positions on half of the head, float32, a pack of odd documents
        _rotary("rotary-grad-f32", 5003, H=12, Hk=4, d=64, dim=32, dtype="f32", interleaved=True, inverse=True,
                where="pack"),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.65:
        dtype = "bf16" if rng.random() < 0.75 else "f32"
        rows = _log_uniform(rng, 1, 32768 if dtype == "bf16" else 6000)
        kind = rng.random()
        if kind < 0.3:
            docs = _pack(rng, rows)
        else:  # one document, or a few of any shape
            parts, left = [], rows
            for _ in range(1 if kind < 0.75 else rng.randint(2, 6)):
                size = rng.randint(1, left)
                ref = rng.choice([0, size, rng.randint(0, size), rng.randint(0, size)])
                parts.append(f"{ref}+{size - ref}")
                left -= size
                if not left:
                    break
            docs = " ".join(parts)
        case = _backward("", docs, n=128 if rng.random() < 0.5 else _log_uniform(rng, 1, 4096),
                         H=_log_uniform(rng, 1, 12), d=rng.choice([64, 128, 128]), dtype=dtype,
                         bidir=rng.random() < 0.3)
        largest = _pairs(listed()[3]) * 10 * 128
        while _pairs(case) * case["H"] * case["d"] > largest and case["H"] > 1:
            case["H"] -= 1
    else:
        d = rng.choice([64, 128])
        H = _log_uniform(rng, 1, 32)
        scaling = rng.choice(["none", "none", "linear", "ntk", "yarn"])
        case = _rotary("", 1, H=H, Hk=rng.choice([H, max(1, H // 4), 1]), d=d,
                       dim=rng.choice([d, d, d // 2, 2 * rng.randint(2, d // 2)]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                       interleaved=rng.random() < 0.5, inverse=rng.random() < 0.4, fused=rng.random() < 0.4,
                       where=rng.choice(["run", "pack", "steps"]), first=rng.choice([0, _log_uniform(rng, 1, 1 << 24)]),
                       scaling=scaling, factor=1.0 if scaling == "none" else rng.uniform(1.5, 32.0))
        most = 32768 * 20 * 128 // ((H + case["Hk"]) * d * (2 if case["dtype"] == "f32" else 1))
        case["rows"] = _log_uniform(rng, 1, min(65536, most))
    del case["name"]
    return case


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rotary":
        rows, heads = case["rows"], case["H"] + case["Hk"]
        # every element read and written once, the positions read once;
        # 6 operations a pair and head, the angle's cosine and sine once a pair and row
        return {"bytes": rows * heads * case["d"] * size * 2 + 4 * rows,
                "flops": rows * (case["dim"] // 2) * (6 * heads + 40)}
    rows, H, d = _documents(case["docs"])[0][-1], case["H"], case["d"]
    # dO, Q, K, V, O and lse read, dQ, dK, dV written; five products over the visible pairs
    return {"bytes": rows * H * (8 * d * size + 4), "flops": 10 * d * H * _pairs(case)}


# ------------------------------------------------------------------ inputs

def _visible(rows, keys, ref, n, bidir):
    i, j = rows[:, None], keys[None, :]
    vis = (j <= i) & ((i < ref) | (j < ref) | (j > i - n))
    return vis | ((i < ref) & (j < ref)) if bidir else vis


def _blocks(case, most):
    """Query blocks of each document and the keys that they can reach:
    (rows of the pack, keys of the pack, visible pairs); a block's scores hold at most `most` elements."""
    cu, refs = _documents(case["docs"])
    for i, ref in enumerate(refs):
        a, size = cu[i], cu[i + 1] - cu[i]
        step = max(16, most // (case["H"] * size))
        for r0 in range(0, size, step):
            r1 = min(size, r0 + step)
            k1 = max(r1, ref) if case["bidir"] else r1
            yield (slice(a + r0, a + r1), slice(a, a + k1),
                   _visible(torch.arange(r0, r1, device="cuda"), torch.arange(k1, device="cuda"), ref, case["n"],
                            case["bidir"]))


def _inv_freq(case):
    """theta_i of each pair in 64 bits, and the factor on cosine and sine."""
    r, base, f = case["dim"], 10000.0, case["factor"]
    if case["scaling"] == "ntk":  # a larger base: the slowest pair is slowed by f, the fastest is kept
        base *= f ** (r / (r - 2))
    theta = [base ** (-2.0 * i / r) for i in range(r // 2)]
    if case["scaling"] == "linear":
        theta = [t / f for t in theta]
    if case["scaling"] == "yarn":
        # pairs that turn more than 32 times over the original 32768 positions
        # are kept, those below one turn are slowed by f, a ramp between
        def pair(turns):
            return r * math.log(32768 / (2 * math.pi * turns)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), r - 1)
        ramp = [min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0) for i in range(r // 2)]
        theta = [t * (1 - w) + t / f * w for t, w in zip(theta, ramp)]
    return theta, (0.1 * math.log(f) + 1.0 if case["scaling"] == "yarn" and f > 1 else 1.0)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if case["op"] == "rotary":
        rows, H, Hk, d = case["rows"], case["H"], case["Hk"], case["d"]
        if case["fused"]:  # queries, keys and values as one projection leaves them: [rows, H + 2 Hk, d]
            qkv = normal(rows, H + 2 * Hk, d).to(dt)
            Q, K = qkv[:, :H], qkv[:, H:H + Hk]
        else:
            Q, K = normal(rows, H, d).to(dt), normal(rows, Hk, d).to(dt)
        pos = torch.arange(rows, device="cuda")
        if case["where"] == "pack":     # documents of 700 rows, each from its first position on
            pos = pos % 700
        elif case["where"] == "steps":  # each row is the newest token of a document of its own
            pos = torch.randint(0, 20000, (rows,), generator=g, device="cuda")
        state = {"case": case, "Q": Q, "K": K, "positions": (pos + case["first"]).to(torch.int32)}
        if own:
            from reference_sliding_window_b200 import Rotary
            state["rotary"] = Rotary(d, rotary_dim=case["dim"], interleaved=case["interleaved"],
                                     scaling=None if case["scaling"] == "none" else case["scaling"],
                                     factor=case["factor"], original_length=32768)
        else:
            theta, state["mscale"] = _inv_freq(case)
            state["theta"] = torch.tensor(theta, dtype=torch.float64, device="cuda")
        return state

    cu, refs = _documents(case["docs"])
    L, H, d = cu[-1], case["H"], case["d"]
    # heads from diffuse to peaked, as trained ones are
    gain = 1.0 + 3.0 * torch.arange(H, device="cuda")[None, :, None] / H
    Q, K, V, dO = (normal(L, H, d) * gain).to(dt), normal(L, H, d).to(dt), normal(L, H, d).to(dt), normal(L, H, d).to(dt)
    # what the forward pass left behind
    O = torch.empty_like(Q)
    lse = torch.empty(H, L, device="cuda")
    for rows, keys, vis in _blocks(case, 1 << 28):
        S = torch.matmul(Q[rows].float().transpose(0, 1), K[keys].float().permute(1, 2, 0)) / math.sqrt(d)
        S.masked_fill_(~vis, -math.inf)
        top = S.amax(-1, keepdim=True)
        S.sub_(top).exp_()
        total = S.sum(-1, keepdim=True)
        O[rows] = (torch.matmul(S, V[keys].float().transpose(0, 1)) / total).transpose(0, 1).to(dt)
        lse[:, rows] = (top + total.log())[..., 0]
    return {"case": case, "dO": dO, "Q": Q, "K": K, "V": V, "O": O, "lse": lse, "cu": cu, "refs": refs}


# -------------------------------------------------------------- plain forms

def _turned(x, cos, sin, dim, interleaved):
    """Every pair of x's first `dim` elements turned by its angle (cos, sin: [rows, 1, pairs])."""
    y = x.float()
    if interleaved:
        a, b = y[..., 0:dim:2], y[..., 1:dim:2]
        rot = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = y[..., :dim // 2], y[..., dim // 2:dim]
        rot = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((rot, y[..., dim:]), dim=-1).to(x.dtype)


def _plain_rotary(state):
    case = state["case"]
    angle = state["positions"].double()[:, None] * state["theta"]
    cos = (angle.cos() * state["mscale"]).float()[:, None]
    sin = (angle.sin() * state["mscale"]).float()[:, None]
    if case["inverse"]:
        sin = -sin
    return tuple(_turned(state[x], cos, sin, case["dim"], case["interleaved"]) for x in ("Q", "K"))


def _plain_backward(state):
    case = state["case"]
    Q, K, V, dO = (state[x].float().transpose(0, 1) for x in ("Q", "K", "V", "dO"))
    scale = 1.0 / math.sqrt(case["d"])
    delta = (state["O"].float().transpose(0, 1) * dO).sum(-1, keepdim=True)
    lse = state["lse"][..., None]
    dQ, dK, dV = torch.zeros_like(Q), torch.zeros_like(K), torch.zeros_like(V)
    for rows, keys, vis in _blocks(case, 1 << 28):
        q, k, v, g = Q[:, rows], K[:, keys], V[:, keys], dO[:, rows]
        P = (torch.matmul(q, k.transpose(1, 2)) * scale - lse[:, rows]).exp().masked_fill(~vis, 0.0)
        dV[:, keys] += torch.matmul(P.transpose(1, 2), g)
        dS = P * (torch.matmul(g, v.transpose(1, 2)) - delta[:, rows]) * scale
        dQ[:, rows] = torch.matmul(dS, k)
        dK[:, keys] += torch.matmul(dS.transpose(1, 2), q)
    return tuple(x.transpose(0, 1).to(state["Q"].dtype).contiguous() for x in (dQ, dK, dV))


def run(state):
    case = state["case"]
    if not own:
        return _plain_rotary(state) if case["op"] == "rotary" else _plain_backward(state)
    if case["op"] == "rotary":
        return state["rotary"].apply(state["Q"], state["K"], positions=state["positions"], inverse=case["inverse"])
    from reference_sliding_window_b200 import masked_backward, masked_backward_varlen
    args = [state[x] for x in ("dO", "Q", "K", "V", "O", "lse")]
    if len(state["refs"]) == 1:
        return masked_backward(*args, L_m=state["refs"][0], n=case["n"], bidir_prefix=case["bidir"])
    return masked_backward_varlen(*args, state["cu"], state["refs"], case["n"], bidir_prefix=case["bidir"])


# -------------------------------------------------------------------- exact

def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "rotary":
        # complex numbers: a pair is x + iy, a turn is a product with m e^(i angle)
        theta, m = _inv_freq(case)
        sign = -1.0 if case["inverse"] else 1.0
        angle = sign * torch.outer(state["positions"].double(), torch.tensor(theta, dtype=torch.float64, device="cuda"))
        turn = torch.polar(torch.full_like(angle, m), angle)[:, None]
        outs = []
        for x in (state["Q"].double(), state["K"].double()):
            r = case["dim"]
            z = x[..., :r].unflatten(-1, (r // 2, 2) if case["interleaved"] else (2, r // 2))
            z = torch.view_as_real(torch.view_as_complex((z if case["interleaved"] else z.transpose(-1, -2)).contiguous()) * turn)
            z = (z if case["interleaved"] else z.transpose(-1, -2)).flatten(-2)
            outs.append(torch.cat((z, x[..., r:]), dim=-1))
        return tuple(outs)
    # the softmax from its definition, not from lse; its gradient from the
    # probabilities and their derivative's mean, not from O
    Q, K, V, dO = (state[x].double().permute(1, 0, 2).contiguous() for x in ("Q", "K", "V", "dO"))
    gQ, gK, gV = (torch.zeros_like(x) for x in (Q, K, V))
    root = case["d"] ** 0.5
    for rows, keys, vis in _blocks(case, 1 << 26):
        A = torch.einsum("hid,hjd->hij", Q[:, rows], K[:, keys]).div_(root)
        A = torch.softmax(A.masked_fill_(~vis, -math.inf), dim=-1)
        gV[:, keys] += torch.einsum("hij,hid->hjd", A, dO[:, rows])
        gA = torch.einsum("hid,hjd->hij", dO[:, rows], V[:, keys])
        gS = A * (gA - (A * gA).sum(-1, keepdim=True)) / root
        gQ[:, rows] = torch.einsum("hij,hjd->hid", gS, K[:, keys])
        gK[:, keys] += torch.einsum("hij,hid->hjd", gS, Q[:, rows])
    return tuple(x.permute(1, 0, 2).contiguous() for x in (gQ, gK, gV))

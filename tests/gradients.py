"""Plain float64 forms of the attention's gradient and of rotary positions,
with error bounds for the CUDA kernels derived from their roundings.

Bounds (u = half a unit in the last place of the tensors' type relative to the
value, e = 2^-23, which covers rounding and truncating float32 accumulation):
* a float32 dot product over d terms: (d + 8) e sum|terms|;
* the probabilities: relative error pe = (d + 8) e (scale sum|q||k|), twice for
  the forward's lse, plus e |lse| and 2^-20 for the exponentials;
* O (read back for delta): (2u + pe) sum P|v| + u|O| (P and O rounded);
* dS = P (dP - delta): pe |dS| + P (1 + pe) (error of dP + error of delta), and
  u |dS| where it is rounded to the tensors' type for the products; the same
  u P for P;
* each sum over m terms: (m + 8) e sum|terms|, and u |x| for the result.
"""

from __future__ import annotations

import math

import torch

import oracle

E32 = 2.0 ** -23
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def visible(cu, refs, n, bidir=False, device="cpu"):
    return torch.from_numpy(oracle.varlen_mask(cu, refs, n, bidir)).to(device)


def backward(dO, Q, K, V, cu, refs, n, scale=0.0, bidir=False, bounds=True):
    """-> ((dQ, dK, dV), (bounds of each), lse): float64 [L, H, d] each, lse [H, L]."""
    dt = Q.dtype
    vis = visible(cu, refs, n, bidir, Q.device)
    q, k, v, g = (t.double().transpose(0, 1) for t in (Q, K, V, dO))
    d, L = q.shape[-1], q.shape[1]
    sc = scale if scale > 0 else 1.0 / math.sqrt(d)
    S = (q @ k.transpose(1, 2) * sc).masked_fill(~vis, -math.inf)
    lse = torch.logsumexp(S, -1, keepdim=True)
    P = (S - lse).exp()
    O = P @ v
    dP = g @ v.transpose(1, 2)
    delta = (O * g).sum(-1, keepdim=True)
    dS = P * (dP - delta)
    grads = (sc * dS @ k, sc * dS.transpose(1, 2) @ q, P.transpose(1, 2) @ g)
    out = tuple(x.transpose(0, 1) for x in grads)
    if not bounds:
        return out, None, lse[..., 0]
    u = U[dt]
    low = u if dt == torch.bfloat16 else 0.0  # P and dS are rounded to the type of the products
    dot = (d + 8) * E32
    aq, ak, av, ag = q.abs(), k.abs(), v.abs(), g.abs()
    pe = 3 * dot * sc * (aq @ ak.transpose(1, 2)) + 2 * E32 * lse.abs() + 2.0 ** -20
    PV = P @ av
    errO = ((2 * low + 2 * u) * PV) + (P * pe) @ av + (L + 8) * E32 * PV + u * O.abs()
    err_delta = (ag * errO).sum(-1, keepdim=True) + dot * (ag * O.abs()).sum(-1, keepdim=True)
    err_dP = dot * (ag @ av.transpose(1, 2))
    err_dS = pe * dS.abs() + P * (1 + pe) * (err_dP + err_delta) + low * dS.abs() * (1 + pe)
    err_P = P * (pe + low * (1 + pe))
    acc = (L + 8) * E32
    b = (sc * (err_dS + acc * dS.abs()) @ ak,
         sc * (err_dS + acc * dS.abs()).transpose(1, 2) @ aq,
         (err_P + acc * P).transpose(1, 2) @ ag)
    tiny = 1e-30
    return out, tuple((x + 1.01 * u * y.abs() + tiny).transpose(0, 1) for x, y in zip(b, grads)), lse[..., 0]


def assert_gradients(got, want, bounds, what=""):
    for name, x, w, b in zip(("dQ", "dK", "dV"), got, want, bounds):
        x = x.double()
        assert torch.isfinite(x).all(), f"{what}: {name} not finite"
        over = ((x - w).abs() / b).max().item()
        assert over <= 1.0, f"{what}: {name} is {over:.3f} times its error bound"


def thetas(dim, base=10000.0, scaling=None, factor=1.0, original_length=0):
    """The turn per position of each pair, and the factor on the result."""
    if scaling == "ntk":
        base = base * factor ** (dim / (dim - 2))
    th = [base ** (-2 * i / dim) for i in range(dim // 2)]
    if scaling == "linear":
        th = [t / factor for t in th]
    m = 1.0
    if scaling == "yarn":
        def index(turns):  # the pair that makes so many turns over the original length
            return dim * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(index(32)), 0), min(math.ceil(index(1)), dim - 1)
        out = []
        for i, t in enumerate(th):
            slow = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            out.append(slow * t / factor + (1 - slow) * t)
        th, m = out, (1 + 0.1 * math.log(factor) if factor > 1 else 1.0)
    return torch.tensor(th, dtype=torch.float64), m


def rotate(x, positions, theta, m=1.0, interleaved=False, inverse=False):
    """float64 rotary positions of x [rows, heads, d]: every pair times a 2x2 matrix."""
    y = x.double().clone()
    r = 2 * theta.numel()
    a = positions.double()[:, None].to(y.device) * theta.to(y.device) * (-1 if inverse else 1)
    R = m * torch.stack((torch.stack((a.cos(), -a.sin()), -1), torch.stack((a.sin(), a.cos()), -1)), -2)
    i = torch.arange(r // 2, device=y.device)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
    pair = torch.stack((y[..., first], y[..., second]), -1)
    out = torch.einsum("rpab,rhpb->rhpa", R, pair)
    y[..., first], y[..., second] = out[..., 0], out[..., 1]
    return y


def rotary_bound(x, want, m=1.0):
    """Error bound of a turned tensor: cosine and sine within 2^-22 m (angle
    and function rounded to float32), three float32 operations per element,
    one rounding to the type.  An element is bounded through its pair's size,
    at most the head's largest element times sqrt 2."""
    size = m * math.sqrt(2.0) * x.double().abs().amax(-1, keepdim=True)
    return 2.0 ** -21 * size + 1.01 * U[x.dtype] * want.abs()


# Norms.  The bounds above add every rounding at its largest and with one sign,
# so an element of a long sum may be far off within them.  A block's norm may
# not: roundings are independent and as often up as down, so that of a sum of
# rounded terms grows as the root of the sum of their squares.  A rounding to
# half a step, relative error at most u, has a root mean square of at most
# s = u / sqrt 3 (uniform within the half step).
# * The results are rounded once: s |x|.
# * For the products P and dS are rounded to bf16 (low = s), or split for three
#   tf32 products, off by 1.25 2^-20 at most (low = R = 2^-19, which covers the
#   rounding of float32 sums of up to 1000 terms too: sqrt(1000) 2^-24 < 2^-19).
# * Scores and dP are float32 sums of such products: R sqrt(sum of squared terms)
#   each; the exponential and its argument's rounding: 2^-21 of P.
# * delta_i gets one error for all of row i, of variance
#   D_i = sum_c g_ic^2 ((s^2 + R^2) O_ic^2 + sum_j (P_ij v_jc)^2 (P's relative variance)):
#   dQ_i is off by it along sum_j P_ij k_j, dK_j by P_ij of it along q_i.  (The
#   row's lse likewise moves all of its P, by 2^-21 at most here.)
# The norm over a block of 64 rows or more is held to three times its root mean
# square: even where one row's delta carries most of it (a first row of few
# keys), a normal error is beyond that once in 370 times at the variance above,
# which is that of the worst mantissas (half of it on average).
BLOCK = 64
R = 2.0 ** -19


def block_errors(dO, Q, K, V, cu, refs, n, scale=0.0, bidir=False):
    """-> ((dQ, dK, dV), (their errors' root mean square per row and head)):
    float64 [L, H, d] and [L, H]."""
    vis = visible(cu, refs, n, bidir, Q.device)
    d = Q.shape[-1]
    sc = scale if scale > 0 else 1.0 / math.sqrt(d)
    s = U[Q.dtype] / math.sqrt(3.0)
    low = s if Q.dtype == torch.bfloat16 else R
    grads, errors = [], []
    for h in range(Q.shape[1]):
        q, k, v, g = (t[:, h].double() for t in (Q, K, V, dO))
        qq, kk, vv, gg = (t * t for t in (q, k, v, g))
        S = (q @ k.T * sc).masked_fill(~vis, -math.inf)
        lse = torch.logsumexp(S, -1, keepdim=True)
        P = (S - lse).exp()
        O = P @ v
        dS = P * (g @ v.T - (O * g).sum(-1, keepdim=True))
        out = (sc * dS @ k, sc * dS.T @ q, P.T @ g)
        before = (R * sc) ** 2 * (qq @ kk.T) + 2.0 ** -42  # relative variance of P before its rounding
        varP = P * P * (before + low * low)
        D = (gg * ((s * s + R * R) * O * O + varP @ vv)).sum(-1)
        vardS = dS * dS * (before + low * low) + P * P * R * R * (gg @ vv.T)
        var = (sc * sc * (vardS @ kk.sum(-1) + D * (P @ k).square().sum(-1)),
               sc * sc * (vardS.T @ qq.sum(-1) + (P * P).T @ (D * qq.sum(-1))),
               varP.T @ gg.sum(-1))
        grads.append(out)
        errors.append([(a + (s * s + R * R) * x.square().sum(-1)).sqrt() for a, x in zip(var, out)])
    return tuple(torch.stack(x, 1) for x in zip(*grads)), tuple(torch.stack(x, 1) for x in zip(*errors))


def blocks(cu):
    """Runs of at least BLOCK rows of one document (the last takes what is left)."""
    for a, b in zip(cu[:-1], cu[1:]):
        for r in range(a, b - BLOCK + 1, BLOCK):
            yield slice(r, b if b - r < 2 * BLOCK else r + BLOCK)


def assert_block_norms(got, want, errors, cu, what=""):
    for name, x, w, e in zip(("dQ", "dK", "dV"), got, want, errors):
        for rows in blocks(cu):
            err = (x[rows].double() - w[rows]).square().sum((0, 2)).sqrt()
            over = (err / e[rows].square().sum(0).sqrt()).max().item()
            assert over <= 3.0, f"{what}: {name}, rows {rows.start} to {rows.stop}: {over:.2f} times its error"  # (NaN fails too)

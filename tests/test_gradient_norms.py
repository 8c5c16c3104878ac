"""The gradient's error in norm, block by block: bounds in tests/gradients.py,
their teeth on the CPU, and the kernels against them."""

from __future__ import annotations

import math

import pytest
import torch

from reference_sliding_window_b200 import masked_backward_varlen, masked_forward_varlen, synth
from tests import gradients

SHAPES = [  # cu, refs, n, heads, bidirectional prefix
    ([0, 300], [100], 16, 2, False),
    ([0, 300], [100], 16, 2, True),
    ([0, 700], [300], 128, 2, False),
    ([0, 700], [0], 128, 2, False),
    ([0, 3000], [2500], 128, 1, False),
]


def _inputs(L, H, d, dtype, seed):
    Q, K, V = synth.prefill_case(L, H, d, dtype, seed)
    return synth.normal((L, H, d), seed * 11 + 5, dtype), (Q.float() * 1.5).to(Q.dtype), K, V


def _rounded(dO, Q, K, V, cu, refs, n, bidir, window=None, delta_by=1.0, noise=0.0, lost=None):
    """The plain gradient with the bf16 kernel's roundings, and with a mistake:
    another window, delta by a factor, noise on dP, a tile pair left out."""
    seen = gradients.visible(cu, refs, n, bidir)
    used = gradients.visible(cu, refs, window or n, bidir)
    if lost is not None:
        used = used.clone()
        used[lost] = False
    gen = torch.Generator().manual_seed(0)
    sc, outs = 1.0 / math.sqrt(Q.shape[-1]), []

    def low(x):
        return x.to(torch.bfloat16).double()

    for h in range(Q.shape[1]):
        q, k, v, g = (t[:, h].double() for t in (Q, K, V, dO))
        S = q @ k.T * sc
        lse = torch.logsumexp(S.masked_fill(~seen, -math.inf), -1, keepdim=True)
        P = (S - lse).exp()
        O = low(low(P.masked_fill(~seen, 0.0)) @ v)
        P = P.masked_fill(~used, 0.0)
        dP = g @ v.T
        dP *= 1 + noise * torch.randn(dP.shape, generator=gen, dtype=torch.float64)
        dS = P * (dP - delta_by * (O * g).sum(-1, keepdim=True))
        outs.append((low(sc * low(dS) @ k), low(sc * low(dS).T @ q), low(low(P).T @ g)))
    return tuple(torch.stack(x, 1) for x in zip(*outs))


@pytest.mark.parametrize("cu,refs,n,H,bidir", [SHAPES[0], SHAPES[1], SHAPES[3], SHAPES[4]])
def test_norms_have_teeth(cu, refs, n, H, bidir):
    """A few percent off, one key more or fewer in the window, a tile left out: each breaks the bound."""
    case = (*_inputs(cu[-1], H, 128, "bf16", seed=cu[-1] + H), cu, refs, n)
    want, errors = gradients.block_errors(*case, bidir=bidir)
    right = _rounded(*case, bidir)
    gradients.assert_block_norms(right, want, errors, cu)
    lost = (slice(128, 256), slice(0, 128)) if cu[-1] < 1000 else (slice(2688, 2816), slice(1280, 1408))

    def breaks(got, which=(0, 1, 2)):
        for i in which:
            with pytest.raises(AssertionError):
                gradients.assert_block_norms(got[i:i + 1], want[i:i + 1], errors[i:i + 1], cu)

    breaks([x * 0.98 for x in right])
    breaks(_rounded(*case, bidir, delta_by=0.95), (0, 1))
    breaks(_rounded(*case, bidir, noise=0.03), (0, 1))
    breaks(_rounded(*case, bidir, window=n + 1))
    breaks(_rounded(*case, bidir, window=n - 1))
    breaks(_rounded(*case, bidir, lost=lost))
    breaks([torch.zeros_like(x) for x in right])
    breaks([x * math.nan for x in right])


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cu,refs,n,H,bidir", SHAPES + [
    ([0, 2000], [0], 1000, 2, False),              # windows over many tiles
    ([0, 1283, 1360, 2900], [400, 77, 900], 100, 2, True),
    ([0, 700, 701, 1500, 2111], [288, 1, 799, 30], 128, 3, False),
])
def test_gradient_in_norm(cu, refs, n, H, bidir, dtype, d):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    dO, Q, K, V = (t.cuda() for t in _inputs(cu[-1], H, d, dtype, seed=cu[-1] + H))
    O, lse = masked_forward_varlen(Q, K, V, cu, refs, n, bidir_prefix=bidir, return_lse=True)
    got = masked_backward_varlen(dO, Q, K, V, O, lse, cu, refs, n, bidir_prefix=bidir)
    want, errors = gradients.block_errors(dO, Q, K, V, cu, refs, n, bidir=bidir)
    gradients.assert_block_norms(got, want, errors, cu, f"{cu} {refs} {n}")

"""CPU tests of the plain gradient and rotary forms that the GPU tests compare
with, and of the host side of their entry points: sizes, plans and refusals."""

from __future__ import annotations

import ctypes as C
import math

import numpy as np
import pytest
import torch

import oracle
from reference_sliding_window_b200 import (Rotary, RSWAError, _native, document_positions, masked_attention,
                                           masked_attention_varlen, masked_backward, masked_forward, synth)
from tests import gradients


@pytest.mark.parametrize("cu,refs,n,bidir,scale", [
    ([0, 9], [4], 2, False, 0.0),
    ([0, 9], [4], 3, True, 0.3),
    ([0, 1, 6, 13], [1, 0, 7], 2, False, 0.0),
])
def test_plain_gradient_matches_differences(cu, refs, n, bidir, scale):
    """Central differences of the oracle's forward, every input element of one head."""
    L, d, h = cu[-1], 3, 1e-5
    rng = np.random.default_rng(L + n)
    X = [rng.standard_normal((L, 1, d)) for _ in range(3)]
    G = rng.standard_normal((L, 1, d))
    got, _, _ = gradients.backward(torch.from_numpy(G), *map(torch.from_numpy, X), cu, refs, n, scale, bidir, bounds=False)

    def f(x):
        return float((oracle.masked_forward_varlen(*x, cu, refs, n, scale=scale, bidir_prefix=bidir) * G).sum())

    for which in range(3):
        for i in range(L):
            for c in range(d):
                hi, lo = [x.copy() for x in X], [x.copy() for x in X]
                hi[which][i, 0, c] += h
                lo[which][i, 0, c] -= h
                # truncation of order h^2, cancellation of order 1e-16 / h
                assert abs((f(hi) - f(lo)) / (2 * h) - got[which][i, 0, c].item()) < 1e-8


def test_error_bounds_have_teeth():
    """A window one key short or one long breaks the bound on spiked queries."""
    cu, refs, n = [0, 60], [20], 8
    Q, K, V = synth.prefill_case(60, 1, 64, "bf16", seed=3)
    Q = synth.spike_packed_queries(Q, K, [(40, 33), (45, 37)])
    dO = synth.normal((60, 1, 64), 8, "bf16")
    want, bounds, _ = gradients.backward(dO, Q, K, V, cu, refs, n)
    gradients.assert_gradients([w.to(torch.bfloat16) for w in want], want, bounds)
    for wrong in (n - 1, n + 1):
        other, _, _ = gradients.backward(dO, Q, K, V, cu, refs, wrong, bounds=False)
        with pytest.raises(AssertionError):
            gradients.assert_gradients(other, want, bounds)


def test_plain_rotary_properties():
    """A turn keeps pair lengths, its inverse undoes it, and products of turned
    vectors depend on the distance of their positions alone."""
    x = torch.randn(5, 2, 64, dtype=torch.float64)
    th, _ = gradients.thetas(32)
    pos = torch.tensor([0, 1, 7, 100, 12345])
    for inter in (False, True):
        y = gradients.rotate(x, pos, th, interleaved=inter)
        assert torch.equal(y[0], x[0]) and torch.equal(y[..., 32:], x[..., 32:])
        assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1), rtol=1e-12)
        assert torch.allclose(gradients.rotate(y, pos, th, interleaved=inter, inverse=True), x, atol=1e-12)
        a, b = (gradients.rotate(t, pos + s, th, interleaved=inter) for t, s in ((x, 0), (x, 50)))
        a2, b2 = (gradients.rotate(t, pos + 999 + s, th, interleaved=inter) for t, s in ((x, 0), (x, 50)))
        assert torch.allclose((a * b).sum(-1), (a2 * b2).sum(-1), atol=1e-9)


@pytest.mark.parametrize("dim,base,scaling,factor,original", [
    (128, 10000.0, None, 1.0, 0), (64, 500000.0, None, 7.0, 0), (2, 10000.0, None, 1.0, 0), (50, 10000.0, "linear", 4.0, 0),
    (64, 10000.0, "ntk", 8.0, 0), (128, 10000.0, "yarn", 8.0, 32768), (32, 10000.0, "yarn", 1.0, 2048),
    (6, 10000.0, "yarn", 40.0, 8),
])
def test_rotary_plan_holds_the_turns(dim, base, scaling, factor, original):
    r = Rotary(128, rotary_dim=dim, base=base, scaling=scaling, factor=factor, original_length=original)
    th, m = gradients.thetas(dim, base, scaling, factor, original)
    assert abs(r.mscale - m) <= 2.0 ** -24 * m
    for i in range(64):
        want = th[i].item() / (2 * math.pi) * 2.0 ** 64 if i < dim // 2 else 0
        # the powers of two libraries agree to a few units of 2^-53; the plan
        # holds the integer part, which is off by less than one
        assert abs(r._plan.turn[i] - want) <= 2.0 ** -50 * want + 1


def test_rotary_plan_refusals():
    for kw in (dict(d=80), dict(d=64, rotary_dim=65), dict(d=64, rotary_dim=31), dict(d=64, rotary_dim=0),
               dict(d=64, rotary_dim=128), dict(d=64, base=1.0), dict(d=64, base=float("nan")),
               dict(d=64, base=float("inf")), dict(d=64, scaling="linear", factor=0.5),
               dict(d=64, scaling="ntk", factor=float("inf")), dict(d=64, scaling="ntk", factor=2.0, rotary_dim=2),
               dict(d=64, scaling="ntk", factor=1e300, base=1e300),
               dict(d=64, scaling="yarn", factor=2.0), dict(d=64, scaling="yarn", factor=float("nan"), original_length=9)):
        with pytest.raises(RSWAError):
            Rotary(**kw)
    with pytest.raises(ValueError, match="scaling"):
        Rotary(64, scaling="other")
    with pytest.raises(ValueError, match="CUDA"):
        Rotary(64).apply(torch.zeros(3, 2, 64))


def test_a_plan_needs_the_library_alone(monkeypatch):
    def missing():
        raise ImportError("no binding")
    monkeypatch.setattr(_native, "binding", missing)
    r = Rotary(64, scaling="linear", factor=2.0)
    assert r.mscale == 1.0 and r._plan.turn[0] > 0
    with pytest.raises(ImportError, match="no binding"):
        r.apply(torch.zeros(3, 2, 64))


def test_host_tensors_are_refused():
    x, lse = torch.zeros(4, 1, 64), torch.zeros(1, 4)
    with pytest.raises(ValueError, match="CUDA"):
        masked_backward(x, x, x, x, x, lse, L_m=2, n=1)
    with pytest.raises(ValueError, match="CUDA"):
        masked_forward(x, x, x, L_m=2, n=1, return_lse=True)
    with pytest.raises(ValueError, match="CUDA"):
        masked_attention(x, x, x, L_m=2, n=1)
    with pytest.raises(ValueError, match="rotary"):
        masked_attention(x, x, x, L_m=2, n=1, positions=torch.arange(4))
    with pytest.raises(ValueError, match="rotary"):
        masked_attention_varlen(x, x, x, [0, 4], [2], 1, positions=torch.arange(4))


def test_document_positions():
    assert document_positions([0, 1, 4, 6], "cpu").tolist() == [0, 0, 1, 2, 0, 1]
    assert document_positions([0, 2], "cpu").dtype == torch.int32
    for bad in ([0], [1, 3], [0, 2, 2]):
        with pytest.raises(ValueError):
            document_positions(bad, "cpu")


@pytest.fixture()
def mem():
    buf = C.create_string_buffer(1 << 16)
    return buf, (C.cast(buf, C.c_void_p).value + 4095) // 4096 * 4096


def _ints(*x):
    return (C.c_int32 * len(x))(*x)


def test_backward_refuses_bad_arguments_before_device(mem):
    # Every call fails the host checks, so nothing is launched.
    _, p = mem
    lib = _native.lib()
    L, H, d = 4, 1, 64
    t = 4 * 64 * 4  # bytes of a tensor

    def call(dO=p, Q=p + t, K=p + 2 * t, V=p + 3 * t, O=p + 4 * t, lse=p + 5 * t, dQ=p + 6 * t, dK=p + 7 * t,
             dV=p + 8 * t, cu=(0, 4), refs=(2,), n_docs=None, n=2, H=H, d=d, dtype=_native.F32, scale=0.0, flags=0,
             ws=p + 9 * t, ws_bytes=1 << 14):
        return lib.rswa_masked_backward(dO, Q, K, V, O, lse, dQ, dK, dV, _ints(*cu), _ints(*(refs or (0,))),
                                        len(refs) if n_docs is None else n_docs, n, H, d, dtype, scale, flags, ws,
                                        ws_bytes, None)

    for name in ("dO", "Q", "K", "V", "O", "lse", "dQ", "dK", "dV", "ws"):
        assert call(**{name: None}) == _native.ERR_ARG
        assert call(**{name: p + 4}) == _native.ERR_ARG
    assert call(n_docs=0) == _native.ERR_ARG
    assert call(cu=(1, 4)) == _native.ERR_ARG
    assert call(cu=(0, 4, 4), refs=(1, 0)) == _native.ERR_ARG
    assert call(cu=(0, 4, 3), refs=(1, 0)) == _native.ERR_ARG
    assert call(refs=(5,)) == _native.ERR_ARG
    assert call(refs=(-1,)) == _native.ERR_ARG
    assert call(n=0) == _native.ERR_ARG
    assert call(H=0) == _native.ERR_ARG
    assert call(flags=2) == _native.ERR_ARG
    assert call(d=80) == _native.ERR_UNSUPPORTED
    assert call(dtype=2) == _native.ERR_UNSUPPORTED
    assert call(scale=float("nan")) == _native.ERR_ARG
    assert call(scale=float("inf")) == _native.ERR_ARG
    assert call(cu=(0, 1 << 30)) == _native.ERR_ARG
    for out in ("dQ", "dK", "dV"):  # a gradient over an input, over another gradient, over the workspace
        for other in range(10):
            if other != {"dQ": 6, "dK": 7, "dV": 8}[out]:
                assert call(**{out: p + other * t}) == _native.ERR_ARG
                assert "overlaps" in lib.rswa_last_error().decode()
    assert call(ws=p + 3 * t + 16, ws_bytes=1 << 10) == _native.ERR_ARG
    assert call(ws_bytes=16) == _native.ERR_ARG
    assert "needed" in lib.rswa_last_error().decode()


def test_backward_workspace_bytes():
    lib = _native.lib()

    def ws(cu, refs, n=128, H=10, d=128, dtype=_native.BF16, flags=0):
        return lib.rswa_masked_backward_workspace_bytes(_ints(*cu), _ints(*refs), len(refs), n, H, d, dtype, flags)

    # the row statistics, 8 bytes per row and head and a tile of rows beyond
    assert ws([0, 100], [50]) >= 10 * 228 * 8
    assert ws([0, 32768], [12832]) < 1 << 28
    assert ws([0, 32768], [12832], H=1) < 1 << 30
    assert ws([0, 100], [101]) == 0
    assert ws([0, 100], [50], d=96) == 0
    assert ws([0, 100], [50], n=0) == 0
    assert ws([0, 100], [50], flags=4) == 0
    # the largest window is the full causal mask
    assert ws([0, 5000], [100], n=2 ** 31 - 1) == ws([0, 5000], [100], n=5000)


def test_forward_lse_refuses_bad_arguments_before_device(mem):
    _, p = mem
    f = _native.lib().rswa_masked_forward_lse
    cu, refs = _ints(0, 4), _ints(2)
    assert f(p, p, p, p, None, cu, refs, 1, 2, 1, 64, _native.F32, 0.0, 0, None) == _native.ERR_ARG
    assert f(p, p, p, p, p + 4, cu, refs, 1, 2, 1, 64, _native.F32, 0.0, 0, None) == _native.ERR_ARG
    assert f(None, p, p, p, p, cu, refs, 1, 2, 1, 64, _native.F32, 0.0, 0, None) == _native.ERR_ARG
    assert f(p, p, p, p, p, cu, _ints(5), 1, 2, 1, 64, _native.F32, 0.0, 0, None) == _native.ERR_ARG


def test_rotary_refuses_bad_arguments_before_device(mem):
    _, p = mem
    lib = _native.lib()
    plan = Rotary(64)._plan
    t = 4 * 2 * 64 * 4  # bytes of [4][2][64] float32

    def call(plan=plan, Q=p, qs=128, H=2, Qo=p + t, qos=128, K=p + 2 * t, ks=128, Hk=2, Ko=p + 3 * t, kos=128,
             pos=None, first=0, rows=4, dtype=_native.F32):
        return lib.rswa_rotary_apply(plan, Q, qs, H, Qo, qos, K, ks, Hk, Ko, kos, pos, first, rows, dtype, 0, None)

    assert call(plan=None) == _native.ERR_ARG
    assert call(plan=_native.RotaryPlan()) == _native.ERR_ARG
    for name in ("Q", "Qo", "K", "Ko"):
        assert call(**{name: None}) == _native.ERR_ARG
        assert call(**{name: p + 4}) == _native.ERR_ARG
    for name in ("qs", "qos", "ks", "kos"):
        assert call(**{name: 127}) == _native.ERR_ARG
        assert call(**{name: 130}) == _native.ERR_ARG  # not a multiple of 16 bytes
        assert call(**{name: 0}) == _native.ERR_ARG
    assert call(rows=0) == _native.ERR_ARG
    assert call(H=0) == _native.ERR_ARG
    assert call(Hk=-1) == _native.ERR_ARG
    assert call(dtype=5) == _native.ERR_UNSUPPORTED
    assert call(first=-1) == _native.ERR_ARG
    assert call(first=2 ** 31 - 3) == _native.ERR_ARG
    assert call(pos=p + 2) == _native.ERR_ARG
    # a result over another tensor, in place with another stride, a shifted overlap
    assert call(Qo=p + 2 * t) == _native.ERR_ARG
    assert call(Ko=p + t) == _native.ERR_ARG
    assert call(Qo=p, qos=256) == _native.ERR_ARG
    assert call(Qo=p + 512) == _native.ERR_ARG
    # rows of one fused buffer: queries, keys; a result over half of the keys
    assert call(Q=p, qs=512, K=p + 512, ks=512, Qo=p + 768, qos=512) == _native.ERR_ARG
    assert lib.rswa_rotary_step(None, plan, p, p, p, p) == _native.ERR_ARG

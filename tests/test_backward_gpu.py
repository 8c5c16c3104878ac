"""GPU tests of the teacher-forced attention's gradient against the plain
float64 form, element by element within bounds derived from the kernels'
roundings (tests/gradients.py)."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from reference_sliding_window_b200 import (RSWA, Rotary, RSWAError, document_positions, masked_attention,
                                           masked_attention_varlen, masked_backward, masked_backward_varlen,
                                           masked_forward, masked_forward_varlen, synth, _native)
from tests import gradients
from tests.gradients import assert_gradients

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def _inputs(L, H, d, dtype, seed, gain=1.5):
    Q, K, V = (t.cuda() for t in synth.prefill_case(L, H, d, dtype, seed))
    dO = synth.normal((L, H, d), seed * 11 + 5, dtype).cuda()
    return dO, (Q.float() * gain).to(Q.dtype), K, V


def _check(dO, Q, K, V, cu, refs, n, scale=0.0, bidir=False, what=""):
    O, lse = masked_forward_varlen(Q, K, V, cu, refs, n, scale=scale, bidir_prefix=bidir, return_lse=True)
    got = masked_backward_varlen(dO, Q, K, V, O, lse, cu, refs, n, scale=scale, bidir_prefix=bidir)
    torch.cuda.synchronize()
    want, bounds, want_lse = gradients.backward(dO, Q, K, V, cu, refs, n, scale, bidir)
    # the row's sum in float32 and its logarithm; scores within (d + 8) 2^-23 of their terms' size
    size = (Q.double().abs() * 1.0).norm(dim=-1).amax() * K.double().norm(dim=-1).amax()
    assert (lse.double() - want_lse).abs().max().item() <= 2.0 ** -23 * ((Q.shape[-1] + 8) * size.item() + Q.shape[0])
    assert_gradients(got, want, bounds, what)
    return got


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L,L_m,n,H,bidir", [
    (1, 1, 1, 1, False),
    (1, 0, 3, 2, False),
    (2, 1, 1, 1, False),
    (63, 20, 5, 1, False),
    (64, 64, 4, 2, False),       # all prefix: plain causal
    (65, 0, 1, 1, False),        # a window of one
    (127, 50, 8, 3, True),
    (128, 128, 16, 1, True),     # full attention
    (129, 1, 128, 2, False),
    (300, 100, 16, 2, False),
    (300, 100, 16, 2, True),
    (520, 129, 1, 3, False),
    (700, 300, 128, 2, False),
    (700, 0, 128, 2, False),     # the plain window
    (700, 0, 200, 1, False),     # windows that reach over two and three tiles
    (640, 384, 260, 1, False),
    (640, 384, 5, 2, True),      # L_m on a tile boundary
    (900, 100, 2 ** 31 - 1, 1, False),  # window wider than the sequence: full causal
])
def test_gradient_every_element(L, L_m, n, H, bidir, dtype, d):
    _check(*_inputs(L, H, d, dtype, seed=L + H), [0, L], [L_m], n, bidir=bidir, what=f"{L} {L_m} {n}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cu,refs,n,bidir", [
    ([0, 300, 428, 956, 1127], [100, 128, 0, 171], 16, False),
    ([0, 384, 700], [200, 300], 8, True),
    ([0, 256, 640, 1024], [3, 129, 384], 5, False),
    ([0, 1, 2, 3, 200, 201], [1, 0, 1, 77, 1], 7, True),
    ([0, 5, 133, 200, 201, 500], [5, 60, 0, 1, 288], 16, False),
])
def test_gradient_of_packs(cu, refs, n, bidir, dtype, d):
    dO, Q, K, V = _inputs(cu[-1], 2, d, dtype, seed=cu[-1] + n)
    _check(dO, Q, K, V, cu, refs, n, bidir=bidir)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 128)])
def test_gradient_of_spiked_queries(dtype, d):
    """Queries spiked on the mask's edges: one key more or less moves the gradient by far more than the bound."""
    L, L_m, n = 600, 200, 130
    dO, Q, K, V = _inputs(L, 2, d, dtype, seed=9)
    probes = [(i, j) for i in (200, 255, 256, 329, 330, 331, 383, 384, 512, 599)
              for j in (i,)] + [(i, i - n + 1) for i in (329, 330, 385, 513, 598)] + \
             [(i, i - n) for i in (340, 386, 514)] + [(i, L_m - 1) for i in (201, 450)] + [(130, 130), (131, 0)]
    seen, keep = set(), []
    for i, j in probes:
        if i not in seen and 0 <= j <= i:
            seen.add(i)
            keep.append((i, j))
    Q = synth.spike_packed_queries(Q, K, keep, gain=2.0)
    _check(dO, Q, K, V, [0, L], [L_m], n)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
@pytest.mark.parametrize("scale", [0.02, 0.5])
def test_gradient_with_a_scale(scale, dtype, d):
    _check(*_inputs(333, 2, d, dtype, seed=4, gain=1.0), [0, 333], [120], 40, scale=scale)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cu,refs,n,bidir", [
    ([0, 1], [1], 7, False),
    ([0, 1], [1], 7, True),
    ([0, 1, 2, 3], [0, 1, 0], 128, False),
    ([0, 300], [0], 1, False),   # a window of one and no prefix
])
def test_rows_of_one_key_have_no_score_gradient(cu, refs, n, bidir, dtype, d):
    """P = 1 whatever the score: dQ and dK are 0, not the rounding of dS."""
    dO, Q, K, V = _inputs(cu[-1], 3, d, dtype, seed=11)
    dQ, dK, _ = _check(dO, Q, K, V, cu, refs, n, bidir=bidir)
    assert not dQ.any() and not dK.any()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cu,refs,n,bidir", [
    ([0, 300, 301, 500], [100, 1, 0], 16, False),
    ([0, 2, 300], [2, 290], 16, False),
    ([0, 130, 300, 430], [1, 0, 0], 5, True),   # a bidirectional prefix of one row, none
    ([0, 3000], [2500], 128, False),            # tiles whose sums are split (with one head)
])
def test_a_document_s_first_row_has_no_score_gradient(cu, refs, n, bidir, dtype, d):
    """It sees itself alone, in a document of any shape: its dQ is 0, and its
    dO moves nothing but dV."""
    H = 1 if cu[-1] == 3000 else 3
    dO, Q, K, V = _inputs(cu[-1], H, d, dtype, seed=15)
    O, lse = masked_forward_varlen(Q, K, V, cu, refs, n, bidir_prefix=bidir, return_lse=True)
    dQ, dK, dV = masked_backward_varlen(dO, Q, K, V, O, lse, cu, refs, n, bidir_prefix=bidir)
    assert not dQ[cu[:-1]].any()
    dO[cu[:-1]] *= 8.0
    other = masked_backward_varlen(dO, Q, K, V, O, lse, cu, refs, n, bidir_prefix=bidir)
    assert torch.equal(dQ, other[0]) and torch.equal(dK, other[1])
    assert not torch.equal(dV, other[2])


def test_a_bidirectional_prefix_gives_the_first_row_its_gradient():
    for dtype, d in (("bf16", 64), ("bf16", 128), ("f32", 64)):
        dQ, _, _ = _check(*_inputs(400, 2, d, dtype, seed=16), [0, 150, 400], [2, 200], 16, bidir=True)
        assert dQ[[0, 150]].any(-1).all()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 128)])
def test_few_heads_and_long_sequences_split_their_sums(dtype, d):
    """One head: tiles with many partners are cut into shares whose sums are joined."""
    _check(*_inputs(3000, 1, d, dtype, seed=6), [0, 3000], [2500], 128)
    _check(*_inputs(2900, 1, d, dtype, seed=7), [0, 100, 2900], [64, 130], 64, bidir=True)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_pack_of_very_many_documents(dtype, d):
    """More work entries than one launch takes: each document is at least a query tile and a key tile."""
    rng = np.random.default_rng(3)
    cu, refs = [0], []
    for size in rng.integers(1, 7, size=700).tolist() + [200]:
        refs.append(int(rng.integers(0, size + 1)))
        cu.append(cu[-1] + size)
    _check(*_inputs(cu[-1], 1, d, dtype, seed=17), cu, refs, 3, bidir=True)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 128)])
def test_two_calls_at_once(dtype, d):
    """Calls on two streams that overlap on the GPU, each with its own workspace."""
    args = []
    for seed in (51, 52):
        dO, Q, K, V = _inputs(2000, 4, d, dtype, seed=seed)
        O, lse = masked_forward(Q, K, V, L_m=700, n=64, return_lse=True)
        args.append((dO, Q, K, V, O, lse))
    want = [masked_backward(*a, L_m=700, n=64) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    got = [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(masked_backward(*args[i], L_m=700, n=64))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            for x, y in zip(g, want[i]):
                assert torch.equal(x, y)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_gradient_repeats_bit_for_bit_and_per_document(dtype, d):
    cu, refs, n = [0, 700, 1001], [288, 30], 128
    dO, Q, K, V = _inputs(cu[-1], 3, d, dtype, seed=12)
    O, lse = masked_forward_varlen(Q, K, V, cu, refs, n, return_lse=True)
    assert torch.equal(O, masked_forward_varlen(Q, K, V, cu, refs, n))
    a = masked_backward_varlen(dO, Q, K, V, O, lse, cu, refs, n)
    junk = torch.full((1 << 24,), float("nan"), device="cuda")  # noqa: F841 (freed memory that a workspace reuses)
    del junk
    b = masked_backward_varlen(dO, Q, K, V, O, lse, cu, refs, n, out=tuple(torch.full_like(Q, float("nan")) for _ in range(3)))
    for x, y in zip(a, b):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 128)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_documents_do_not_touch_each_other(bad, dtype, d):
    """Infinities and NaN in one document leave the others' gradients as they were."""
    cu, refs, n = [0, 200, 330, 475], [60, 130, 10], 16
    dO, Q, K, V = _inputs(cu[-1], 2, d, dtype, seed=13)
    O, lse = masked_forward_varlen(Q, K, V, cu, refs, n, return_lse=True)
    clean = masked_backward_varlen(dO, Q, K, V, O, lse, cu, refs, n)
    for t in (dO, Q, K, V, O):
        t[200:330] = bad
    lse[:, 200:330] = bad
    got = masked_backward_varlen(dO, Q, K, V, O, lse, cu, refs, n)
    for x, y in zip(got, clean):
        assert torch.equal(x[:200], y[:200]) and torch.equal(x[330:], y[330:])


@pytest.mark.parametrize("d", [64, 128])
def test_short_documents_whose_tiles_come_from_memory_do_not_touch_each_other(d):
    """Thousands of documents shorter than a tile, ten heads, several times
    what L2 holds, and NaN in the dO of every second one: the clean ones keep
    their bits, call after call.  Every document's tiles reach over the next
    one's rows, and each of an item's loads may land at any time."""
    H, n, docs = 10, 40, 2400 if d == 64 else 1200
    rng = np.random.default_rng(d)
    sizes = rng.integers(1, 128, size=docs)
    cu = [0] + np.cumsum(sizes).tolist()
    refs = [int(rng.integers(0, s + 1)) for s in sizes]
    g = torch.Generator(device="cuda").manual_seed(d)
    dO, Q, K, V = (torch.randn((cu[-1], H, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(4))
    O, lse = masked_forward_varlen(Q, K, V, cu, refs, n, return_lse=True)
    clean = masked_backward_varlen(dO, Q, K, V, O, lse, cu, refs, n)
    rows = torch.from_numpy(np.repeat(np.arange(docs) % 2 == 0, sizes)).cuda()
    dO[~rows] = float("nan")
    for _ in range(5):
        got = masked_backward_varlen(dO, Q, K, V, O, lse, cu, refs, n)
        for name, x, y in zip(("dQ", "dK", "dV"), got, clean):
            assert torch.equal(x[rows], y[rows]), name


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ctas", [10 ** 6, 1, 40])
def test_rows_of_a_kernel_that_gives_up_are_nan(ctas, d):
    """Waits that run out (injected on the host) leave no row as it was: the
    items that the CTAs held, had taken without starting them, or never took
    are NaN, the others right; split sums too.  The next call is right again."""
    give_up = _native.lib().rswa_testing_backward_give_up
    give_up.argtypes, give_up.restype = [ctypes.c_int], None
    rng = np.random.default_rng(ctas)
    short = np.cumsum(rng.integers(1, 200, size=400)).tolist()
    for cu, refs, H in (([0, 3000], [2500], 1),        # every item in shares
                        ([0, 700, 1001], [288, 30], 3),  # fewer items than CTAs
                        ([0] + short, [0] * len(short), 4)):  # many short items a CTA, two launches
        dO, Q, K, V = _inputs(cu[-1], H, d, "bf16", seed=33)
        O, lse = masked_forward_varlen(Q, K, V, cu, refs, 64, return_lse=True)
        want = masked_backward_varlen(dO, Q, K, V, O, lse, cu, refs, 64)
        out = tuple(torch.full_like(Q, 7.0) for _ in range(3))
        try:
            give_up(ctas)
            got = masked_backward_varlen(dO, Q, K, V, O, lse, cu, refs, 64, out=out)
        finally:
            give_up(0)
        torch.cuda.synchronize()
        assert any(x.isnan().any() for x in got)
        for x, y in zip(got, want):
            if ctas >= 1000:
                assert x.isnan().all()
            else:
                assert torch.where(x.isnan(), y, x).equal(y)
        for x, y in zip(masked_backward_varlen(dO, Q, K, V, O, lse, cu, refs, 64), want):
            assert torch.equal(x, y)


def test_gradient_32k_sampled():
    """The 32768-row teacher-forced sequence (12832 reference rows, 10 heads,
    bf16): rows of dQ, dK and dV on the mask's edges and at random, against
    float64 sums over all their partners."""
    L, L_m, n, H, d = 32768, 12832, 128, 10, 128
    g = torch.Generator(device="cuda").manual_seed(5)
    dO, Q, K, V = (torch.randn((L, H, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(4))
    O, lse = masked_forward(Q, K, V, L_m=L_m, n=n, return_lse=True)
    dQ, dK, dV = masked_backward(dO, Q, K, V, O, lse, L_m=L_m, n=n)
    rng = np.random.default_rng(5)
    rows = sorted({0, 1, 127, 128, L_m - 1, L_m, L_m + 1, L_m + n, L - n, L - 1} | set(rng.integers(0, L, 16).tolist()))
    idx = torch.arange(L, device="cuda")
    for h in (0, 9):
        q, k, v, do = (t[:, h].double() for t in (Q, K, V, dO))
        o, ls = O[:, h].double(), lse[h].double()
        delta = (o * do).sum(-1)
        for r in rows:
            # dQ of row r, over its keys
            vis = (idx <= r) & ((r < L_m) | (idx < L_m) | (idx > r - n))
            p = torch.where(vis, (k @ q[r] / d ** 0.5 - ls[r]).exp(), 0.0)
            ds = p * (v @ do[r] - delta[r])
            # bf16 dS and result, and as much again for delta's O and the float32 sums
            tol = 2.0 ** -7 * (ds.abs() @ k.abs() + p @ k.abs() * (o[r].abs() @ do[r].abs())) / d ** 0.5 + 2.0 ** -7 * 1e-3
            assert ((dQ[r, h].double() - ds @ k / d ** 0.5).abs() <= tol).all(), f"dQ {r} {h}"
            # dK, dV of row r, over its queries
            vis = (r <= idx) & ((idx < L_m) | (r < L_m) | (r > idx - n))
            p = torch.where(vis, (q @ k[r] / d ** 0.5 - ls).exp(), 0.0)
            ds = p * (do @ v[r] - delta)
            tol = 2.0 ** -7 * (ds.abs() @ q.abs() + (p * (o * do).abs().sum(-1)) @ q.abs()) / d ** 0.5 + 2.0 ** -7 * 1e-3
            assert ((dK[r, h].double() - ds @ q / d ** 0.5).abs() <= tol).all(), f"dK {r} {h}"
            tol = 2.0 ** -7 * (p @ do.abs()) + 2.0 ** -7 * 1e-3
            assert ((dV[r, h].double() - p @ do).abs() <= tol).all(), f"dV {r} {h}"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_training_step_of_a_pack(dtype):
    """Rotary positions, attention over a pack, a loss and its gradient back
    to the unturned Q, K and V, as a training step uses them together."""
    cu, refs, n, H, d = [0, 333, 471], [120, 40], 50, 2, 128
    dO, Q, K, V = _inputs(cu[-1], H, d, dtype, seed=21, gain=1.0)
    rot = Rotary(d, rotary_dim=96)
    for t in (Q, K, V):
        t.requires_grad_()
    O = masked_attention_varlen(Q, K, V, cu, refs, n, rotary=rot)
    O.backward(dO)
    pos = document_positions(cu).cpu()
    th, _ = gradients.thetas(96)
    q, k, v = (t.detach().double().cpu().requires_grad_() for t in (Q, K, V))
    # the plain form in float64, through the same turns by differentiation
    qr, kr = _turn(q, pos, th), _turn(k, pos, th)
    vis = gradients.visible(cu, refs, n)
    S = torch.einsum("ihd,jhd->hij", qr, kr) / d ** 0.5
    o = torch.einsum("hij,jhd->ihd", S.masked_fill(~vis, -float("inf")).softmax(-1), v)
    o.backward(dO.double().cpu())
    # turned Q, K and the gradients on either side of the turn back are rounded
    # to the type: relative errors of a few u in norm, sums of independent signs
    u = gradients.U[Q.dtype]
    for x, y in ((O, o), (Q.grad, q.grad), (K.grad, k.grad), (V.grad, v.grad)):
        err = (x.detach().double().cpu() - y.detach()).norm() / y.norm()
        assert err.item() <= 8 * u + 2.0 ** -20


def _turn(x, pos, theta):
    half = theta.numel()
    a = (pos.double()[:, None] * theta)[:, None]
    x0, x1 = x[..., :half], x[..., half:2 * half]
    return torch.cat((x0 * a.cos() - x1 * a.sin(), x1 * a.cos() + x0 * a.sin(), x[..., 2 * half:]), -1)


def test_attention_of_one_document_and_expanded_gradients():
    L, L_m, n, H, d = 150, 60, 20, 2, 64
    dO, Q, K, V = _inputs(L, H, d, "f32", seed=22)
    for t in (Q, V):
        t.requires_grad_()
    O = masked_attention(Q, K, V, L_m=L_m, n=n, bidir_prefix=True)
    O.sum().backward()  # an expanded gradient of ones
    ones = torch.ones_like(O)
    want, bounds, _ = gradients.backward(ones, Q.detach(), K, V.detach(), [0, L], [L_m], n, bidir=True)
    assert K.grad is None
    assert_gradients((Q.grad, V.grad), (want[0], want[2]), (bounds[0], bounds[2]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_off_a_16_byte_address(dtype):
    """The gradient of a part of a concatenation starts anywhere."""
    L, L_m, n, H, d = 70, 20, 9, 2, 64
    dO, Q, K, V = _inputs(L, H, d, dtype, seed=27)
    leaves = [t.clone().requires_grad_() for t in (Q, K, V)]
    rot = Rotary(d)
    pad = torch.zeros(1, device="cuda", dtype=Q.dtype)

    def grads(off):
        q, k = rot(*leaves[:2])
        q, k = ((torch.cat([pad, t.flatten()])[1:].clone().view_as(t) if off else t) for t in (q, k))
        O = masked_attention(q, k, leaves[2], L_m=L_m, n=n)
        if off:
            loss = (torch.cat([pad, O.flatten()]) * torch.cat([pad, dO.flatten()])).sum()
        else:
            loss = (O * dO).sum()
        return torch.autograd.grad(loss, leaves)

    for x, y in zip(grads(False), grads(True)):
        assert torch.equal(x, y)


def test_backward_on_another_stream_and_captured():
    """On a side stream, and captured once and replayed on new inputs; two
    graphs keep their own workspaces."""
    L, L_m, n, H, d = 400, 150, 33, 2, 128
    dO, Q, K, V = _inputs(L, H, d, "bf16", seed=30)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        O, lse = masked_forward(Q, K, V, L_m=L_m, n=n, return_lse=True)
        first = masked_backward(dO, Q, K, V, O, lse, L_m=L_m, n=n)
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                o, ls = masked_forward(Q, K, V, L_m=L_m, n=n, return_lse=True)
                outs = masked_backward(dO, Q, K, V, o, ls, L_m=L_m, n=n)
            graphs.append((g, outs))
    torch.cuda.current_stream().wait_stream(side)
    for seed in (31, 32):
        for t, x in zip((dO, Q, K, V), _inputs(L, H, d, "bf16", seed=seed)):
            t.copy_(x)
        for g, _ in graphs:
            g.replay()
        O, lse = masked_forward(Q, K, V, L_m=L_m, n=n, return_lse=True)
        want = masked_backward(dO, Q, K, V, O, lse, L_m=L_m, n=n)
        torch.cuda.synchronize()
        for _, outs in graphs:
            for x, y in zip(outs, want):
                assert torch.equal(x, y)
        assert not torch.equal(first[0], want[0])


def _captured_step(seed):
    """Static leaves, and one training step over them (a pack, with positions)."""
    cu, refs, n, d = [0, 150, 333], [90, 40], 25, 64
    dO, Q, K, V = _inputs(cu[-1], 2, d, "bf16", seed=seed)
    leaves = [t.clone().requires_grad_() for t in (Q, K, V)]
    rot, pos = Rotary(d), document_positions(cu)

    def step():
        O = masked_attention_varlen(*(t * 1.0 for t in leaves), cu, refs, n, rotary=rot, positions=pos)
        return torch.autograd.grad((O * dO).sum(), leaves)

    return leaves, dO, step


def test_training_step_captured():
    """Forward and backward in one graph, replayed on new inputs."""
    leaves, dO, step = _captured_step(70)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for seed in (71, 72):
        for t, x in zip((dO, *leaves), _inputs(leaves[0].shape[0], 2, 64, "bf16", seed=seed)):
            t.data.copy_(x)
        g.replay()
        want = step()
        torch.cuda.synchronize()
        for x, y in zip(outs, want):
            assert torch.equal(x, y)


def test_capture_is_refused_while_an_eager_graph_lives():
    """A result kept on the default stream holds the leaves: refused in the
    forward call, before the backward pass could end the process."""
    leaves, _, step = _captured_step(80)
    kept = sum(t.float().sum() for t in leaves)
    side = torch.cuda.Stream()
    rot, a = Rotary(64), torch.zeros(1, device="cuda")
    with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=side):
        a.add_(1)
        with pytest.raises(ValueError, match="default stream"):
            step()
        with pytest.raises(ValueError, match="default stream"):
            rot(leaves[0])
        with pytest.raises(ValueError, match="before the capture"):
            document_positions([0, 3])
        with torch.no_grad():
            rot(leaves[0])
    del kept
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        outs = step()
    g.replay()
    for x, y in zip(outs, step()):
        assert torch.equal(x, y)


def test_decode_after_a_turned_prefill():
    """Prefill with rotary positions, then decode steps that turn q and k at
    the handle's own step, against the packed form of the whole sequence."""
    L_m, n, T0, T, H, d = 90, 8, 11, 24, 2, 128
    L = L_m + T
    Q, K, V = (t.cuda() for t in synth.prefill_case(L, H, d, "f32", seed=40))
    rot = Rotary(d, interleaved=True)
    want = masked_attention(Q, K, V, L_m=L_m, n=n, rotary=rot)
    a = RSWA(L_m, n, H, d, 1, torch.float32)
    got = a.prefill(Q[:L_m + T0].contiguous(), K[:L_m + T0].contiguous(), V[:L_m + T0].contiguous(), L_m, rotary=rot)
    assert torch.equal(got, want[:L_m + T0])
    for t in range(T0, T):
        p = L_m + t  # the row that output t + 1 takes
        o = a.append_decode(K[p:p + 1], V[p:p + 1], Q[p:p + 1], rotary=rot)
        err = (o[0] - want[p]).abs().max() / want[p].abs().max()
        assert err.item() <= 1e-5, f"output {t + 1}"
    a.check()


def test_both_ways_into_the_library_agree():
    """Given results, and documents as an array, take the longer way in."""
    cu, refs, n = [0, 200, 333], [90, 40], 25
    dO, Q, K, V = _inputs(cu[-1], 2, 64, "bf16", seed=60)
    O, lse = masked_forward_varlen(Q, K, V, cu, refs, n, return_lse=True)
    a = masked_backward_varlen(dO, Q, K, V, O, lse, cu, refs, n)
    b = masked_backward_varlen(dO, Q, K, V, O, lse, np.array(cu), np.array(refs), np.int64(n))
    c = masked_backward_varlen(dO, Q, K, V, O, lse, cu, refs, n, out=[torch.empty_like(Q) for _ in range(3)])
    for x, y, z in zip(a, b, c):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_refusals():
    dO, Q, K, V = _inputs(16, 2, 64, "f32", seed=1)
    O, lse = masked_forward(Q, K, V, L_m=4, n=2, return_lse=True)
    ok = dict(L_m=4, n=2)
    with pytest.raises(ValueError):
        masked_backward(dO, Q, K, V, O, lse.T.contiguous(), **ok)
    with pytest.raises(ValueError):
        masked_backward(dO, Q, K, V, O, lse.double(), **ok)
    with pytest.raises(ValueError):
        masked_backward(dO[:8], Q, K, V, O, lse, **ok)
    with pytest.raises(ValueError):
        masked_backward(dO.transpose(0, 1), Q, K, V, O, lse, **ok)
    with pytest.raises(ValueError):
        masked_backward(dO.bfloat16(), Q, K, V, O, lse, **ok)
    with pytest.raises(ValueError):
        masked_backward(dO, Q.half(), K, V, O, lse, **ok)
    with pytest.raises(ValueError):
        masked_backward(dO.cpu(), Q, K, V, O, lse, **ok)
    with pytest.raises(ValueError):
        masked_backward(dO, Q, K, V, O, lse, out=(Q, K), **ok)
    with pytest.raises(RSWAError, match="overlaps"):
        masked_backward(dO, Q, K, V, O, lse, out=(dO, torch.empty_like(Q), torch.empty_like(Q)), **ok)
    with pytest.raises(RSWAError, match="ARG"):
        masked_backward(dO, Q, K, V, O, lse, L_m=17, n=2)
    with pytest.raises(RSWAError, match="ARG"):
        masked_backward(dO, Q, K, V, O, lse, L_m=4, n=0)
    with pytest.raises(ValueError):
        masked_backward_varlen(dO, Q, K, V, O, lse, [0, 8, 15], [1, 1], 2)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_the_largest_tensors(dtype, d):
    """Just under 2^31 elements a tensor: the last document of the pack has the
    bits that it has alone."""
    H, last = 16, 700
    L = (2 ** 31 // d - 1) // H
    if dtype == "f32":
        L //= 4  # (8 tensors of 8.6 GB would do, but take their time)
    cu, refs, n = [0, 100, L - last, L], [50, 0, 288], 128
    g = torch.Generator(device="cuda").manual_seed(1)
    t = [torch.empty((L, H, d), dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device="cuda") for _ in range(4)]
    for x in t:
        for rows in x.split(1 << 18):
            rows.normal_(generator=g)
    dO, Q, K, V = t
    rot = Rotary(d)
    Q, K = rot.apply(Q, K, out=(Q, K))
    O, lse = masked_forward_varlen(Q, K, V, cu, refs, n, return_lse=True)
    got = masked_backward_varlen(dO, Q, K, V, O, lse, cu, refs, n)
    for a, b, ref in ((L - last, L, 288), (0, 100, 50)):
        part = [x[a:b].clone() for x in (dO, Q, K, V, O)]
        alone = masked_forward(*part[1:4], L_m=ref, n=n, return_lse=True)
        assert torch.equal(part[4], alone[0]) and torch.equal(lse[:, a:b], alone[1])
        want = masked_backward(*part, alone[1], L_m=ref, n=n)
        for x, y in zip(got, want):
            assert torch.equal(x[a:b], y)
    # rows of the long window, against its own last rows run alone: dQ alone is whole there
    a, b = L - last - 1280, L - last
    part = [x[a:b].clone() for x in (dO, Q, K, V, O)]
    want = masked_backward(*part, lse[:, a:b].contiguous(), L_m=0, n=n)
    assert (got[0][a + n:b].float() - want[0][n:].float()).abs().max() <= 2.0 ** -6 * want[0].float().abs().max()

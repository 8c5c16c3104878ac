"""GPU tests of rotary positions against the plain float64 form."""

from __future__ import annotations

import copy

import pytest
import torch

from reference_sliding_window_b200 import RSWA, Rotary, RSWAError, synth
from tests import gradients

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def _close(got, x, pos, kw, inverse=False):
    d = x.shape[-1]
    dim = kw.get("rotary_dim", d)
    th, m = gradients.thetas(dim, kw.get("base", 10000.0), kw.get("scaling"), kw.get("factor", 1.0),
                             kw.get("original_length", 0))
    want = gradients.rotate(x.cpu(), pos.cpu(), th, m, kw.get("interleaved", False), inverse)
    err = (got.double().cpu() - want).abs()
    assert (err <= gradients.rotary_bound(x.cpu(), want, m)).all()
    assert torch.equal(got[..., dim:], x[..., dim:])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,dim", [(128, 128), (64, 64), (128, 64), (128, 48), (64, 2), (64, 26), (128, 120), (128, 126), (64, 36)])
def test_layouts_and_parts_of_the_head(d, dim, interleaved, dtype):
    kw = dict(rotary_dim=dim, interleaved=interleaved)
    rot = Rotary(d, **kw)
    for rows, H, Hk in ((1, 1, 1), (37, 5, 3)):
        Q, K = (synth.normal((rows, h, d), rows + h, dtype).cuda() for h in (H, Hk))
        pos = torch.randint(0, 40000, (rows,), dtype=torch.int32, generator=torch.Generator().manual_seed(dim)).cuda()
        for inverse in (False, True):
            q, k = rot.apply(Q, K, positions=pos, inverse=inverse)
            _close(q, Q, pos, kw, inverse)
            _close(k, K, pos, kw, inverse)
        # without positions, from `first` on; queries alone
        q = rot.apply(Q, first=777)
        _close(q, Q, torch.arange(777, 777 + rows), kw)


@pytest.mark.parametrize("kw", [
    dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0), dict(base=500000.0),
    dict(scaling="yarn", factor=8.0, original_length=32768), dict(scaling="yarn", factor=2.5, original_length=2048,
                                                                  rotary_dim=64, interleaved=True),
])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scaled_for_long_contexts(kw, dtype):
    Q = synth.normal((50, 3, 128), 5, dtype).cuda()
    pos = (torch.arange(50, dtype=torch.int32) * 5003).cuda()
    q = Rotary(128, **kw).apply(Q, positions=pos)
    _close(q, Q, pos, kw)


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(interleaved):
    """Angles hold however far the position: a float64 product of position and
    theta is itself off by 2^-53 of 2^31 radians, 2^-22."""
    kw = dict(interleaved=interleaved)
    Q = synth.normal((8, 2, 64), 6, "f32").cuda()
    pos = torch.tensor([0, 1, 2 ** 20 + 1, 2 ** 24 + 1, 2 ** 30 + 3, 2 ** 31 - 1, 123456789, 2 ** 22 - 1], dtype=torch.int32).cuda()
    _close(Rotary(64, **kw).apply(Q, positions=pos), Q, pos, kw)
    last = Rotary(64, **kw).apply(Q, first=2 ** 31 - 8)
    _close(last, Q, torch.arange(2 ** 31 - 8, 2 ** 31), kw)


def test_negative_positions_turn_back():
    Q = synth.normal((4, 2, 64), 7, "f32").cuda()
    pos = torch.tensor([-1, -100, -(2 ** 31), -12345], dtype=torch.int32).cuda()
    _close(Rotary(64).apply(Q, positions=pos), Q, pos, {})


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [128, 100])
def test_slices_of_a_fused_projection_and_in_place(dtype, dim):
    rows, H, Hk, d = 301, 4, 2, 128
    rot = Rotary(d, rotary_dim=dim)
    qkv = synth.normal((rows, H + 2 * Hk, d), 8, dtype).cuda()
    Q, K = qkv[:, :H], qkv[:, H:H + Hk]
    q, k = rot.apply(Q, K)
    assert q.is_contiguous() and k.is_contiguous()
    q2, k2 = rot.apply(Q.contiguous(), K.contiguous())
    assert torch.equal(q, q2) and torch.equal(k, k2)
    _close(q, Q, torch.arange(rows), dict(rotary_dim=dim))
    keep = qkv.clone()
    out = rot.apply(Q, K, out=(Q, K))  # in place, inside the wider rows
    assert out[0].data_ptr() == Q.data_ptr()
    assert torch.equal(qkv[:, :H], q) and torch.equal(qkv[:, H:H + Hk], k)
    assert torch.equal(qkv[:, H + Hk:], keep[:, H + Hk:])  # the values beside them are left alone
    # into other slices of wide rows
    wide = torch.zeros_like(qkv)
    rot.apply(keep[:, :H], keep[:, H:H + Hk], out=(wide[:, Hk:Hk + H], wide[:, :Hk]))
    assert torch.equal(wide[:, Hk:Hk + H], q) and torch.equal(wide[:, :Hk], k)
    assert not wide[:, H + Hk:].any()


def test_many_rows():
    """More rows than threads resident at once, each thread with several heads."""
    Q, K = torch.randn(70001, 3, 64, device="cuda"), torch.randn(70001, 1, 64, device="cuda")
    q, k = Rotary(64).apply(Q, K)
    _close(q[-50:], Q[-50:], torch.arange(70001)[-50:], {})
    _close(k[::997], K[::997], torch.arange(70001)[::997], {})


def test_gradient_is_the_inverse_turn():
    """<dY, R dX> = <R^T dY, dX> against float64 differences of the plain form."""
    rot = Rotary(64, scaling="yarn", factor=4.0, original_length=1024)
    th, m = gradients.thetas(64, scaling="yarn", factor=4.0, original_length=1024)
    x, gy = torch.randn(9, 2, 64), torch.randn(9, 2, 64)
    gx = rot.apply(gy.cuda(), inverse=True).double().cpu()
    for _ in range(5):
        v = torch.randn(9, 2, 64, dtype=torch.float64)
        f = [(gradients.rotate(x.double() + s * 1e-3 * v, torch.arange(9), th, m) * gy.double()).sum() for s in (1, -1)]
        diff = ((f[0] - f[1]) / 2e-3).item()  # linear: exact up to rounding
        assert abs((gx * v).sum().item() - diff) <= 2.0 ** -20 * (gy.double().norm() * v.norm() * m).item()


@pytest.mark.parametrize("pair", [False, True])
def test_differentiable_call_and_copies(pair):
    rot = copy.deepcopy(Rotary(64, rotary_dim=40, interleaved=True, scaling="linear", factor=3.0))
    th, m = gradients.thetas(40, scaling="linear", factor=3.0)
    x = [torch.randn(7, h, 64, device="cuda", requires_grad=True) for h in ((3, 2) if pair else (3,))]
    pos = torch.arange(7, dtype=torch.int32, device="cuda") * 11
    y = rot(*x, positions=pos)
    y = y if pair else (y,)
    g = [torch.randn_like(t).transpose(0, 1).contiguous().transpose(0, 1) for t in y]  # not contiguous
    torch.autograd.backward(y, g)
    for t, o, go in zip(x, y, g):
        _close(o.detach(), t.detach(), pos, dict(rotary_dim=40, interleaved=True, scaling="linear", factor=3.0))
        want = gradients.rotate(go.cpu(), pos.cpu(), th, m, True, True)
        assert ((t.grad.double().cpu() - want).abs() <= gradients.rotary_bound(go.cpu(), want, m)).all()
    with pytest.raises(ValueError):
        rot(torch.zeros(3, 2, 32, device="cuda"))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_both_ways_into_the_library_agree(dtype):
    """A tensor subclass and given results take the longer way in."""
    class Sub(torch.Tensor):
        pass
    Q, K = (synth.normal((9, h, 64), h, dtype).cuda() for h in (3, 1))
    rot = Rotary(64)
    a = rot.apply(Q, K, first=5)
    b = rot.apply(Q.as_subclass(Sub), K, first=5)
    c = rot.apply(Q, K, first=5, out=(torch.empty_like(Q), torch.empty_like(K)))
    for x, y, z in zip(a, b, c):
        assert torch.equal(x, torch.as_tensor(y)) and torch.equal(x, z)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_step_of_a_handle(dtype):
    """rotate() follows the handle's device-side step, ragged, also captured and replayed."""
    refs, n, H, d, T = [40, 13, 27], 8, 2, 64, 12
    case = synth.decode_case(3, H, d, refs, n, T, dtype, seed=50)
    rot = Rotary(d)
    a = RSWA(case.L_m_cap, n, H, d, 3, synth.torch_dtype(dtype))
    a.load_reference(case.K_ref.cuda(), case.V_ref.cuda(), refs)
    k, v, q = (t.cuda() for t in (case.k, case.v, case.q))
    qs, ks, vs, os_ = q[0].clone(), k[0].clone(), v[0].clone(), torch.empty_like(q[0])
    for t in range(T // 2):
        pos = torch.tensor(refs) + t
        qt, kt = a.rotate(rot, q[t], k[t])
        _close(qt, q[t], pos, {})
        _close(kt, k[t], pos, {})
        a.append_decode(k[t], v[t], q[t], rotary=rot)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qt, kt = a.rotate(rot, qs, ks)
        a.append_decode(kt, vs, qt, out=os_)
    for t in range(T // 2, T):
        qs.copy_(q[t])
        ks.copy_(k[t])
        g.replay()
        torch.cuda.synchronize()
        _close(qt, q[t], torch.tensor(refs) + t, {})
    assert a.step_count() == [T] * 3
    # in place
    x, y = q[0].clone(), k[0].clone()
    a.rotate(rot, x, y, out=(x, y))
    _close(x, q[0], torch.tensor(refs) + T, {})
    a.check()


def test_refusals():
    rot = Rotary(64)
    Q = torch.zeros(4, 2, 64, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (torch.zeros(4, 2, 32, device="cuda"), Q[0], Q.half(), Q.transpose(1, 2), Q.expand(4, 2, 64)[:, :, ::2]):
        with pytest.raises(ValueError):
            rot.apply(bad)
    with pytest.raises(ValueError):
        rot.apply(Q, positions=pos.long())
    with pytest.raises(ValueError):
        rot.apply(Q, positions=pos[:3])
    with pytest.raises(ValueError):
        rot.apply(Q, positions=pos.cpu())
    with pytest.raises(ValueError):
        rot.apply(Q, Q.bfloat16())
    with pytest.raises(ValueError):
        rot.apply(Q, Q[:3])
    with pytest.raises(ValueError):
        rot.apply(Q, out=torch.zeros(4, 3, 64, device="cuda"))
    with pytest.raises(RSWAError, match="ARG"):
        rot.apply(Q[:1].expand(4, 2, 64))            # every row the same memory
    with pytest.raises(RSWAError, match="ARG"):
        rot.apply(torch.zeros(0, 2, 64, device="cuda"))
    with pytest.raises(RSWAError, match="overlap"):
        rot.apply(Q, Q.clone(), out=(Q, Q))          # both results in one place
    a = RSWA(8, 4, 2, 64, 1, torch.float32)
    x = torch.zeros(1, 2, 64, device="cuda")
    with pytest.raises(RSWAError, match="STATE"):
        a.rotate(rot, x, x.clone())
    with pytest.raises(RSWAError, match="ARG"):
        a.rotate(Rotary(128), x, x.clone())


@pytest.mark.parametrize("dim,interleaved", [(2, False), (6, True)])
def test_more_than_2_32_threads(dim, interleaved):
    """Element by element (rotary dims below a vector), in place, over a tensor of
    9 10^9 elements: the rows have the values that they have in a small call."""
    rows = 140_000_003
    rot = Rotary(64, rotary_dim=dim, interleaved=interleaved)
    Q = torch.empty((rows, 1, 64), dtype=torch.bfloat16, device="cuda")
    for part in Q.split(1 << 24):
        part.normal_(generator=torch.Generator(device="cuda").manual_seed(part.storage_offset() & 0xffff))
    some = [(0, 300), (rows // 2, rows // 2 + 300), ((1 << 27) - 150, (1 << 27) + 150), (rows - 300, rows)]
    want = [rot.apply(Q[a:b].clone(), first=a) for a, b in some]
    rot.apply(Q, out=Q)
    for (a, b), w in zip(some, want):
        assert torch.equal(Q[a:b], w)

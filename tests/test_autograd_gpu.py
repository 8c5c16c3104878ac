"""GPU tests of the differentiable calls beyond one plain backward pass: second
derivatives, transforms, compilation, recomputation, gradients asked of some."""

from __future__ import annotations

import pytest
import torch
from torch.autograd import forward_ad
from torch.utils.checkpoint import checkpoint

from reference_sliding_window_b200 import Rotary, masked_attention, masked_attention_varlen, synth
from tests import gradients

pytestmark = pytest.mark.gpu

L, H, D = 150, 2, 64


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def _qkv(dtype="f32"):
    return tuple(t.cuda() for t in synth.prefill_case(L, H, D, dtype, 3))


def _attend(q, k, v, rotary=None):
    return masked_attention(q, k, v, L_m=60, n=20, rotary=rotary)


def _calls():
    rot = Rotary(D)
    return {"plain": _attend, "turned": lambda q, k, v: _attend(q, k, v, rot),
            "pack": lambda q, k, v: masked_attention_varlen(q, k, v, [0, 70, L], [30, 0], 20, rotary=rot)}


@pytest.mark.parametrize("name", ["plain", "turned", "pack"])
@pytest.mark.parametrize("which", [0, 1, 2])
def test_a_second_derivative_of_the_attention_raises(name, which):
    """A gradient penalty: the part that cannot be differentiated is not dropped
    from the sum of both, whichever input is asked for."""
    x = list(_qkv())
    x[which].requires_grad_()
    loss = _calls()[name](*x).square().sum()
    g, = torch.autograd.grad(loss, x[which], create_graph=True)
    assert torch.equal(g, torch.autograd.grad(loss, x[which], retain_graph=True)[0])
    with pytest.raises(RuntimeError, match="once differentiable"):
        torch.autograd.grad(loss + g.square().sum(), x[which], retain_graph=True)
    with pytest.raises(RuntimeError, match="once differentiable"):
        (loss + g.square().sum()).backward()


@pytest.mark.parametrize("name", ["plain", "turned"])
def test_a_second_derivative_raises_where_the_first_depends_on_the_inputs_alone(name):
    """The output's gradient is constant: dQ depends on Q through what was saved of it."""
    q, k, v = _qkv()
    q.requires_grad_()
    loss = _calls()[name](q, k, v).sum()
    g, = torch.autograd.grad(loss, q, create_graph=True)
    with pytest.raises(RuntimeError, match="once differentiable"):
        torch.autograd.grad(loss + g.square().sum(), q)


@pytest.mark.parametrize("pair", [False, True])
def test_a_turn_is_differentiable_twice(pair):
    """loss = |R x|^2 m^-2 / 2 per element weighed with w: gradients by the plain form in float64."""
    kw = dict(rotary_dim=40, interleaved=True)
    rot, (th, m) = Rotary(D, **kw), gradients.thetas(40)
    xs = [torch.randn(9, h, D, device="cuda", requires_grad=True) for h in ((3, 2) if pair else (3,))]
    ws = [torch.randn_like(x) for x in xs]
    pos = torch.arange(9, dtype=torch.int32, device="cuda") * 7
    ys = rot(*xs, positions=pos)
    ys = ys if pair else (ys,)
    first = torch.autograd.grad(sum((w * y ** 3).sum() for w, y in zip(ws, ys)), xs, create_graph=True)
    got = torch.autograd.grad(sum(g.square().sum() for g in first), xs)

    def turn(x, inverse=False):
        r = gradients.rotate(x.detach().cpu(), pos.cpu(), th, m, True, inverse)
        return r

    for x, w, g1, g2 in zip(xs, ws, first, got):
        y, wd = turn(x), w.double().cpu()
        f1 = turn(3 * wd * y * y, True)          # R^T of the loss's gradient
        f2 = turn(6 * wd * y * turn(2 * f1), True)  # and R^T diag(6 w y) R of |f1|^2's
        for g, f in ((g1, f1), (g2, f2)):
            # float32: three turns and products, a few relative roundings each
            assert (g.double().cpu() - f).norm() <= 2.0 ** -19 * f.norm()


def test_transforms_that_the_calls_do_not_have_raise():
    q, k, v = _qkv()
    rot = Rotary(D)
    two = [torch.stack([t, t]) for t in (q, k, v)]
    with pytest.raises(RuntimeError):
        torch.vmap(_attend)(*two)
    with pytest.raises(RuntimeError):
        torch.vmap(rot)(two[0])
    with pytest.raises(RuntimeError):
        torch.vmap(lambda x: rot.apply(x))(two[0])
    with pytest.raises(RuntimeError):
        torch.func.grad(lambda x: _attend(x, k, v).sum())(q)
    with forward_ad.dual_level():
        for call in (lambda x: _attend(x, k, v), rot):
            with pytest.raises((RuntimeError, NotImplementedError)):
                call(forward_ad.make_dual(q, q))
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", ["plain", "turned"])
def test_compiled_functions_run_the_calls_as_they_are(name):
    call = _calls()[name]

    def step(q, k, v):
        return call(q * 1.0, k, v) * 2.0

    leaves = [t.requires_grad_() for t in _qkv("bf16")]
    outs = [(o, torch.autograd.grad(o.float().square().sum(), leaves))
            for o in (step(*leaves), torch.compile(step, backend="eager")(*leaves))]
    assert torch.equal(outs[0][0], outs[1][0])
    for x, y in zip(outs[0][1], outs[1][1]):
        assert torch.equal(x, y)


@pytest.mark.parametrize("name", ["plain", "turned", "pack"])
def test_recomputed_in_the_backward_pass(name):
    call = _calls()[name]
    leaves = [t.requires_grad_() for t in _qkv("bf16")]
    want = torch.autograd.grad(call(*leaves).float().square().sum(), leaves)
    got = torch.autograd.grad(checkpoint(call, *leaves, use_reentrant=False).float().square().sum(), leaves)
    for x, y in zip(got, want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("name", ["plain", "turned"])
def test_gradients_of_some_inputs(name):
    call = _calls()[name]
    x = _qkv("bf16")
    want = torch.autograd.grad(call(*(t.requires_grad_() for t in x)).float().square().sum(), x)
    for which in range(3):
        y = [t.detach().clone() for t in x]
        y[which].requires_grad_()
        call(*y).float().square().sum().backward()
        assert [t.grad is None for t in y] == [i != which for i in range(3)]
        assert torch.equal(y[which].grad, want[which])

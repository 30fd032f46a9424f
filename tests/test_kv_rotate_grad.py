"""Gradients of kv_rotate through autograd: the transposed map, rounded once to BF16 (tolerances as in test_kv_rotate.py)."""
import pytest
import torch

import kv_more_reference as M
import kv_reference as R
from bit_routed_expert_gb300 import kv_rotate, rope_turns


def test_outputs_of_the_caller_are_refused_where_gradients_are_wanted():
    turns, pos = torch.zeros(8, dtype=torch.int64), torch.zeros(2, dtype=torch.int32)
    plain, wants = (torch.zeros(2, 2, 64, dtype=torch.bfloat16, requires_grad=r) for r in (False, True))
    for q, k, kw in ((wants, None, dict(q_out=plain)), (plain, wants, dict(k_out=plain)), (wants, plain, dict(q_out=plain, k_out=plain))):
        with pytest.raises(ValueError, match="gradients"):
            kv_rotate(q, k, pos, turns, **kw)
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):   # (refused later, for another reason)
            kv_rotate(q, k, pos, turns, **kw)


def near(got, want, size):
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -21 * size + 2.0 ** -133
    return bool(((got.cpu().double() - want).abs() <= tol).all())


@pytest.mark.gpu
@pytest.mark.parametrize("D,P,offset,inter,backward", [(64, 32, 0, False, False), (128, 32, 64, True, False), (64, 12, 8, False, True),
                                                       (96, 1, 5, True, False)])
@pytest.mark.parametrize("of_q,of_k", [(True, True), (True, False), (False, True)])
def test_gradients(cuda_dev, D, P, offset, inter, backward, of_q, of_k):
    T, Hq, Hk, gain = 21, 6, 2, 1.25
    turns, _ = rope_turns(2 * P)
    pos = torch.arange(T, dtype=torch.int32) * 77777
    pos[::5] = -1
    qkv = R.rows(1, T, Hq + 2 * Hk, D).to(cuda_dev)
    q, k = qkv[:, :Hq].detach().requires_grad_(of_q), qkv[:, Hq:Hq + Hk].detach().requires_grad_(of_k)
    args = pos.to(cuda_dev), turns.to(cuda_dev), gain, offset, inter, backward
    qo, ko = kv_rotate(q, k, *args)
    with torch.no_grad():
        q0, k0 = kv_rotate(q, k, *args)
    assert torch.equal(qo, q0) and torch.equal(ko, k0) and not q0.requires_grad
    assert (qo.requires_grad, ko.requires_grad) == (of_q, of_k)
    wq, wk = R.rows(2, T, Hq, D), R.rows(3, T, Hk, D)
    loss = [(y, w.to(cuda_dev)) for y, w in ((qo, wq), (ko, wk)) if y.requires_grad]
    torch.autograd.backward(*zip(*loss))
    for x, w, needs in ((q, wq, of_q), (k, wk, of_k)):
        assert (x.grad is not None) == needs
        if needs:
            assert near(x.grad, *M.rotate(w, pos, [int(t) % 2 ** 64 for t in turns], gain, offset, inter, not backward))


@pytest.mark.gpu
def test_through_a_projection(cuda_dev):
    """Queries and keys as slices of a product, one of the outputs unused, a gradient that is one number for all channels."""
    T, Hq, Hk, D = 9, 4, 2, 64
    turns, pos = rope_turns(D, device=cuda_dev)[0], torch.arange(T, dtype=torch.int32, device=cuda_dev)
    w = (R.rows(1, 32, (Hq + Hk) * D).to(cuda_dev)).requires_grad_()
    x = R.rows(2, T, 32).to(cuda_dev)
    qk = (x @ w).view(T, Hq + Hk, D)
    qo, _ = kv_rotate(qk[:, :Hq], qk[:, Hq:], pos, turns)
    qo.sum().backward()
    ones, _ = kv_rotate(torch.ones_like(qo), None, pos, turns, backward=True)
    ones = ones.view(T, -1).double()
    want, size = x.double().T @ ones, x.double().abs().T @ ones.abs()   # FP32 sums of nine products, rounded to BF16
    assert bool(((w.grad[:, :Hq * D].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * size).all())
    assert not bool(w.grad[:, Hq * D:].any())
    a = qk.detach().requires_grad_()   # no key, and a gradient of a gradient
    y, none = kv_rotate(a, None, pos, turns)
    assert none is None
    v = torch.ones_like(y).requires_grad_()
    g, = torch.autograd.grad(y, a, v, create_graph=True)
    back, = torch.autograd.grad(g, v, R.rows(5, T, Hq + Hk, D).to(cuda_dev))
    assert torch.equal(back, kv_rotate(R.rows(5, T, Hq + Hk, D).to(cuda_dev), None, pos, turns)[0])


@pytest.mark.gpu
def test_positions_changed_before_the_backward_pass_are_noticed(cuda_dev):
    turns, pos = rope_turns(64, device=cuda_dev)[0], torch.arange(3, dtype=torch.int32, device=cuda_dev)
    q = R.rows(1, 3, 2, 64).to(cuda_dev).requires_grad_()
    y, _ = kv_rotate(q, None, pos, turns)
    pos += 1
    with pytest.raises(RuntimeError, match="modified"):
        y.sum().backward()


@pytest.mark.gpu
def test_forward_and_backward_in_a_graph_and_on_a_stream(cuda_dev):
    """(Nothing that autograd recorded outside of the capture may live on through it: PyTorch would join that one's stream.)"""
    turns, pos = rope_turns(64, device=cuda_dev)[0], torch.arange(40, dtype=torch.int32, device=cuda_dev)
    q = R.rows(1, 40, 6, 64).to(cuda_dev).requires_grad_()
    w = R.rows(2, 40, 6, 64).to(cuda_dev)

    def both(stream=None):
        y, _ = kv_rotate(q, None, pos, turns, stream=stream)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        g, = torch.autograd.grad(y, q, w)
        return y.detach(), g
    want, grad = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(side)
    assert torch.equal(got[0], want) and torch.equal(got[1], grad)
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, g = both()
    pos += 5
    graph.replay()
    want, grad = both()
    assert torch.equal(y, want) and torch.equal(g, grad)

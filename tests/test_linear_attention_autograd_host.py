"""The autograd bindings of the linear-attention operators without a GPU: the library's
calls are replaced by recorders, everything around them runs as it is."""
import pytest
import torch

from selective_state_space_mamba3_gb300 import autograd

ROWS, HEADS, WIDTH, ANGLES = 6, 2, 8, 4


@pytest.fixture
def calls(monkeypatch):
    """The library calls made: (name, positional arguments)."""
    made = []
    for name in ("m3_qk_norm_rope", "m3_qk_norm_rope_backward", "m3_linear_attention_forward",
                 "m3_linear_attention_backward"):
        monkeypatch.setattr(autograd.m3, name, lambda *a, n=name: made.append((n, a)))
    for name in ("m3_qk_norm_rope_backward_workspace", "m3_linear_attention_forward_workspace",
                 "m3_linear_attention_backward_workspace"):
        monkeypatch.setattr(autograd.m3, name, lambda cfg: 256)
    return made


def operand(*shape):
    return torch.zeros(*shape or (ROWS, HEADS, WIDTH)).requires_grad_()


def tables():
    return torch.ones(16, ANGLES), torch.zeros(16, ANGLES), torch.zeros(ROWS, dtype=torch.int32)


@pytest.mark.parametrize("which", [0, 1, 2])
def test_tables_written_again_before_the_backward_call_are_an_error(calls, which):
    tabs = tables()
    q, k = autograd.qk_norm_rope(operand(), operand(), None, None, *tabs, ANGLES)
    tabs[which].add_(1)
    with pytest.raises(RuntimeError, match="inplace"):
        (q.sum() + k.sum()).backward()
    assert [n for n, _ in calls] == ["m3_qk_norm_rope"]


@pytest.mark.parametrize("which", ["offsets", "log_decay", "initial_state"])
def test_offsets_and_states_written_again_before_the_backward_call_are_an_error(calls, which):
    t = dict(offsets=torch.tensor([0, 2, 6], dtype=torch.int32), log_decay=torch.zeros(HEADS),
             initial_state=torch.zeros(2, HEADS, WIDTH, WIDTH))
    out = autograd.linear_attention(operand(), operand(), operand(), t["log_decay"], 2, 4,
                                    offsets=t["offsets"], initial_state=t["initial_state"])
    t[which].add_(1)
    with pytest.raises(RuntimeError, match="inplace"):
        out.sum().backward()
    assert [n for n, _ in calls] == ["m3_linear_attention_forward"]


def test_the_adjoints_get_the_forward_calls_operands(calls):
    tabs = tables()
    off = torch.tensor([0, 2, 6], dtype=torch.int32)
    q, k = autograd.qk_norm_rope(operand(), operand(), None, None, *tabs, ANGLES)
    autograd.linear_attention(q, k, operand(), torch.zeros(HEADS), 2, 4, offsets=off).sum().backward()
    assert [n for n, _ in calls] == ["m3_qk_norm_rope", "m3_linear_attention_forward",
                                     "m3_linear_attention_backward", "m3_qk_norm_rope_backward"]
    fwd, bwd = calls[1][1], calls[2][1]
    assert torch.equal(fwd[5], off) and torch.equal(bwd[6], off)
    for a, b in zip(calls[0][1][5:8], calls[3][1][5:8]):
        assert torch.equal(a, b)


def test_an_unused_state_costs_the_adjoint_no_zeros(calls):
    out, fin = autograd.linear_attention(operand(), operand(), operand(), torch.zeros(HEADS), 1, ROWS,
                                         return_state=True)
    out.sum().backward()
    grad_out, grad_final = calls[1][1][1], calls[1][1][8]
    assert grad_out is not None and grad_final is None


def test_outputs_the_loss_does_not_use_have_zero_gradients(calls):
    v = operand()
    _, fin = autograd.linear_attention(operand(), operand(), v, torch.zeros(HEADS), 1, ROWS,
                                       return_state=True)
    fin.sum().backward()
    grad_out, grad_final = calls[1][1][1], calls[1][1][8]
    assert torch.equal(grad_out, torch.zeros_like(v)) and torch.equal(grad_final, torch.ones_like(fin))
    del calls[:]
    q, _ = autograd.qk_norm_rope(operand(), operand(ROWS, 1, WIDTH), None, None, *tables(), ANGLES)
    q.sum().backward()
    dq, dk = calls[1][1][8:10]
    assert torch.equal(dq, torch.ones(ROWS, HEADS, WIDTH))
    assert torch.equal(dk, torch.zeros(ROWS, 1, WIDTH))


@pytest.mark.parametrize("which", [0, 1])
def test_a_gradient_of_the_rotation_tables_is_refused(calls, which):
    tabs = tables()
    tabs[which].requires_grad_()
    with pytest.raises(ValueError, match="tables"):
        autograd.qk_norm_rope(operand(), operand(), None, None, *tabs, ANGLES)
    assert not calls


def test_a_second_derivative_is_refused(calls):
    """The adjoints are no functions of torch: a graph of them would lack their terms."""
    x = operand()
    q, _ = autograd.qk_norm_rope(x, None, None, None, *tables(), ANGLES)
    (g,) = torch.autograd.grad(q.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()
    out = autograd.linear_attention(x, x, x, torch.zeros(HEADS), 1, ROWS)
    (g,) = torch.autograd.grad(out.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()


def test_a_second_derivative_among_other_terms_is_refused(calls):
    x = operand()
    for loss in (lambda y: y.sum(), lambda y: y.square().sum()):
        out = autograd.linear_attention(x, x, x, torch.zeros(HEADS), 1, ROWS)
        (g,) = torch.autograd.grad(loss(out), x, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            (g.square().sum() + x.square().sum()).backward()
        (g,) = torch.autograd.grad(loss(autograd.linear_attention(x, x, x, torch.zeros(HEADS), 1, ROWS)), x)
        assert not g.requires_grad


@pytest.mark.parametrize("default", [torch.float64, torch.bfloat16])
def test_states_are_float32_whatever_the_default_type(calls, default):
    x = operand()  # float32
    torch.set_default_dtype(default)
    try:
        out, fin = autograd.linear_attention(x, x, x, torch.zeros(HEADS, dtype=torch.float32), 1, ROWS,
                                             return_state=True)
    finally:
        torch.set_default_dtype(torch.float32)
    assert out.dtype == fin.dtype == torch.float32

"""The binding's own checks of the linear-attention operators, without a GPU: operands that
say which device they are on, and a library that records what reaches it."""
import pytest
import torch

import selective_state_space_mamba3_gb300 as m3
from selective_state_space_mamba3_gb300 import _binding

ROWS, HEADS, P, N, ANGLES, SLOTS = 6, 2, 8, 16, 4, 5
F, I, U = torch.float32, torch.int32, torch.uint8


class On:
    """A CPU tensor that says it is on a CUDA device."""
    is_cuda = True

    def __init__(self, t, index=0):
        self.t, self.index = t, index

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.index

    @property
    def device(self):
        return torch.device("cuda", self.index)


class Library:
    """Accepts every call and keeps its name."""

    def __init__(self):
        self.made = []

    def __getattr__(self, name):
        return lambda *a: self.made.append(name) or 0


@pytest.fixture
def made(monkeypatch):
    lib = Library()
    types = _binding._torch_types()
    monkeypatch.setattr(_binding, "load_library", lambda: lib)
    # streams and the current device (0) without a CUDA runtime
    monkeypatch.setattr(_binding, "_types", (*types[:3], lambda index: 0, lambda: 0))
    return lib.made


def la_cfg(batch, length, slots=0):
    return m3.LinearAttentionConfig(batch, length, batch * length, HEADS, 1, P, N, slots, 0, 0, 0, 0,
                                    1.0, 0)


ROPE = m3.QkNormRopeConfig(ROWS, HEADS, 1, N, ANGLES, 32, 0, 0, 0, 0, 1e-6, 0)
Q, K, QK, V, S = (ROWS, HEADS, N), (ROWS, 1, N), (ROWS, 1, N), (ROWS, HEADS, P), (2, HEADS, P, N)
TABLES = dict(q_weight=(F, N), k_weight=(F, N), cos=(F, 32, ANGLES), sin=(F, 32, ANGLES),
              positions=(I, ROWS))
WS = dict(ws=(U, 4096))
# call, config, operands in order
CALLS = {
    "rope": (m3.m3_qk_norm_rope, ROPE,
             dict(q=(F, *Q), k=(F, *K), **TABLES, q_out=(F, *Q), k_out=(F, *K))),
    "rope_backward": (m3.m3_qk_norm_rope_backward, ROPE,
                      dict(q=(F, *Q), k=(F, *K), **TABLES, dq_out=(F, *Q), dk_out=(F, *K), dq=(F, *Q),
                           dk=(F, *K), dq_weight=(F, N), dk_weight=(F, N), **WS)),
    "forward": (m3.m3_linear_attention_forward, la_cfg(2, 3),
                dict(q=(F, *QK), k=(F, *QK), v=(F, *V), decay=(F, HEADS), offsets=(I, 3), s0=(F, *S),
                     out=(F, *V), final=(F, *S), **WS)),
    "step": (m3.m3_linear_attention_step, la_cfg(2, 1, SLOTS),
             dict(q=(F, 2, 1, N), k=(F, 2, 1, N), v=(F, 2, HEADS, P), decay=(F, HEADS), slots=(I, 2),
                  state=(F, SLOTS, HEADS, P, N), out=(F, 2, HEADS, P))),
    "backward": (m3.m3_linear_attention_backward, la_cfg(2, 3),
                 dict(dout=(F, *V), q=(F, *QK), k=(F, *QK), v=(F, *V), decay=(F, HEADS),
                      offsets=(I, 3), s0=(F, *S), ds=(F, *S), dq=(F, *QK), dk=(F, *QK), dv=(F, *V),
                      ds0=(F, *S), **WS)),
}
EVERY = [(c, x) for c, (_, _, spec) in CALLS.items() for x in spec]


def call(which, device=0, **other):
    """Makes a call with every operand as it should be, but for `other`."""
    fn, cfg, spec = CALLS[which]
    fn(cfg, *[other[x] if x in other else On(torch.zeros(*shape, dtype=dt), device)
              for x, (dt, *shape) in spec.items()])


@pytest.mark.parametrize("which", CALLS)
def test_calls_as_they_should_be_reach_the_library(which, made):
    call(which)
    assert len(made) == 1


@pytest.mark.parametrize("which,operand", EVERY)
def test_an_operand_on_another_device_is_refused(which, operand, made):
    dt, *shape = CALLS[which][2][operand]
    with pytest.raises(ValueError, match="device"):
        call(which, **{operand: On(torch.zeros(*shape, dtype=dt), 1)})
    with pytest.raises(TypeError):  # not on a GPU
        call(which, **{operand: torch.zeros(*shape, dtype=dt)})
    assert not made


@pytest.mark.parametrize("which", CALLS)
def test_operands_on_a_device_that_is_not_the_current_one_are_refused(which, made):
    """The library launches on the calling thread's current device."""
    with pytest.raises(ValueError, match="current device"):
        call(which, device=1)
    assert not made


@pytest.mark.parametrize("which,operand,shape", [
    ("forward", "s0", (2, HEADS, N, P)), ("forward", "final", (HEADS, 2 * P, N // 2, 2)),
    ("forward", "final", (2, P, N, HEADS)), ("step", "state", (HEADS, SLOTS, P, N)),
    ("backward", "ds", (2, HEADS, N, P)), ("rope", "cos", (ANGLES, 32)),
    ("rope_backward", "sin", (ANGLES, 2, 16))])
def test_another_shape_of_as_many_values_is_refused(which, operand, shape, made):
    with pytest.raises(ValueError, match="shape"):
        call(which, **{operand: On(torch.zeros(*shape))})
    assert not made


@pytest.mark.parametrize("which,operand,dt,shape", [
    ("forward", "s0", F, (2 * HEADS, P, N)), ("forward", "final", F, (2 * HEADS * P * N,)),
    ("forward", "s0", F, (2, HEADS, P * N)), ("backward", "ds", F, (2, 1, HEADS, P, N)),
    ("step", "state", F, (SLOTS, HEADS * P, N)), ("rope", "cos", F, (4, 8, ANGLES)),
    ("rope", "positions", I, (2, ROWS // 2)), ("rope", "q_weight", F, (1, 1, N)),
    ("forward", "decay", F, (1, HEADS, 1, 1)), ("forward", "decay", F, (HEADS,)), ("rope", "sin", F, (32 * ANGLES,))])
def test_the_same_values_in_other_dimensions_pass(which, operand, dt, shape, made):
    """Dimensions merged, split at the front, or of one value: the memory is the same."""
    call(which, **{operand: On(torch.zeros(*shape, dtype=dt))})
    assert len(made) == 1


def uneven(rows):
    """Rows of two heads that do not lie evenly: `rows` of five, three times."""
    return torch.zeros(3, 5, HEADS, N)[:, :rows]


def test_rows_that_are_not_evenly_spaced_are_refused():
    even = torch.zeros(3, 5, HEADS, N)
    assert m3.qk_norm_rope_config(even, even, num_rope_angles=0).q_stride == HEADS * N
    with pytest.raises(TypeError, match="evenly"):
        m3.qk_norm_rope_config(uneven(4), even, num_rope_angles=0)
    with pytest.raises(TypeError, match="evenly"):
        m3.qk_norm_rope_config(even, uneven(4), num_rope_angles=0)
    with pytest.raises(TypeError, match="evenly"):
        m3.qk_norm_rope_config(even, even, num_rope_angles=0, k_out=uneven(4))
    for bad in range(3):
        qkv = [even, even, even]
        qkv[bad] = uneven(4)
        with pytest.raises(TypeError, match="evenly"):
            m3.linear_attention_config(*qkv, batch_size=3, sequence_length=5)


def test_rows_that_differ_from_the_configs_are_refused(made):
    apart = On(torch.zeros(ROWS, 2, HEADS, N)[:, 0])  # evenly spaced, but not as the config says
    with pytest.raises(ValueError, match="stride"):
        call("rope", q=apart)
    with pytest.raises(TypeError, match="evenly"):  # as many rows as the config's, unevenly
        call("rope", q=On(torch.zeros(2, 4, HEADS, N)[:, :3]))
    assert not made

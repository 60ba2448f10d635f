"""Linear attention on the GPU with values far from one: every intermediate has to
fit where its result does. Operands are scaled by a power of two, which commutes with
every rounding in the normal range, so the tolerances are those of linattn_ref."""
import pytest

import linattn_ref as ref
import selective_state_space_mamba3_gb300 as m3
from test_gpu_linear_attention import DTYPES, Problem, bar, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from selective_state_space_mamba3_gb300 import build
    build.build()


def scaled(p, operand, state, exponent):
    """Multiplies one operand and the state that its results add to."""
    f = 2.0 ** exponent
    p.d[operand] *= f
    p.h[operand] *= f
    state *= f


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("exponent", [90, -90])
@pytest.mark.parametrize("decay", [0.0, -0.1, -0.5, -0.51])
@pytest.mark.parametrize("L,N", [(5, 64), (200, 64), (300, 128)])
def test_values_far_from_one(dtype, L, N, decay, exponent):
    p = Problem(1, L, 2, 0, 64, N, dtype, states=True, seed=30 + L, decay=decay)
    scaled(p, "v", p.s0, exponent)
    p.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("exponent", [90, -90])
@pytest.mark.parametrize("decay", [0.0, -0.1, -0.5, -0.51])
def test_gradients_far_from_one(dtype, decay, exponent):
    p = Problem(1, 200, 2, 0, 64, 64, dtype, states=True, seed=31, decay=decay)
    scaled(p, "do", p.ds, exponent)
    for name, a, b in zip(("dq", "dk", "dv", "ds0"), p.backward(), p.ref_backward()):
        assert ref.rel(host(a), b) <= (ref.F32_BAR if name == "ds0" else bar(dtype)), name


@pytest.mark.parametrize("scale", [0.0, 1e-12, 1e12])
@pytest.mark.parametrize("decay", [-0.1, -0.5])
def test_scales_far_from_one(scale, decay):
    """(The states do not see the scale, or only as dout does.)"""
    p = Problem(1, 200, 2, 0, 64, 64, "bf16", states=True, seed=32, decay=decay)
    p.cfg = m3.linear_attention_config(p.d["q"], p.d["k"], p.d["v"], batch_size=1,
                                       sequence_length=200, num_heads=2, scale=scale)
    p.scale = p.cfg.scale
    got = [p.forward()[0], *p.backward()[:3]]
    want = [p.ref_forward()[0], *p.ref_backward()[:3]]
    for name, a, b in zip(("out", "dq", "dk", "dv"), got, want):
        assert ref.rel(host(a), b) <= bar("bf16"), name

"""Linear-attention operators without a GPU: the adjoint formulas against
central differences of the forward statement, and every refusal of the C ABI
(rejected calls enqueue nothing and never follow the fake pointers)."""
import ctypes

import numpy as np
import pytest

import linattn_ref as ref
import selective_state_space_mamba3_gb300 as m3
from selective_state_space_mamba3_gb300 import build as m3build

FAKE, FAKE4 = 0x10000, 0x10004


@pytest.fixture(scope="module")
def lib():
    m3build.build()
    return m3.load_library()


# --- formulas ----------------------------------------------------------------

def numeric(f, x, eps=1e-5):
    g = np.zeros(x.shape)
    for i in np.ndindex(x.shape):
        old = x[i]
        x[i] = old + eps
        hi = f()
        x[i] = old - eps
        lo = f()
        x[i] = old
        g[i] = (hi - lo) / (2 * eps)
    return g


@pytest.mark.parametrize("groups,offsets", [(2, None), (1, [0, 3, 3, 4])])
def test_adjoint_formulas_are_the_derivatives(groups, offsets):
    rng = np.random.default_rng(5)
    B, L = (2, 2) if offsets is None else (3, 4)
    rows, H, P, N = 4, 2, 3, 2
    q, k, v, do = (rng.standard_normal(s) for s in
                   ((rows, groups, N), (rows, groups, N), (rows, H, P), (rows, H, P)))
    s0, ds = rng.standard_normal((B, H, P, N)), rng.standard_normal((B, H, P, N))
    ld = np.array([-0.3, -1.1])

    def loss():
        out, fin = ref.forward(q, k, v, ld, 0.7, B, L, offsets, s0)
        return (out * do).sum() + (fin * ds).sum()

    got = ref.backward(do, q, k, v, ld, 0.7, B, L, offsets, s0, ds)
    for g, x in zip(got, (q, k, v, s0)):
        # the loss is multilinear: central differences are exact up to rounding, 1e-16 / 1e-5
        np.testing.assert_allclose(g, numeric(loss, x), atol=1e-8)


def test_rope_adjoint_formula_is_the_derivative():
    rng = np.random.default_rng(6)
    x, dy, w = rng.standard_normal((3, 2, 7)), rng.standard_normal((3, 2, 7)), rng.uniform(.5, 2, 7)
    ang = rng.uniform(0, 6, (4, 3))
    pos = np.array([3, 0, 9])
    f = lambda: (ref.rope(x, w, np.cos(ang), np.sin(ang), pos, 1e-3) * dy).sum()  # noqa: E731
    dx, dw = ref.rope_backward(x, w, np.cos(ang), np.sin(ang), pos, 1e-3, dy)
    np.testing.assert_allclose(dx, numeric(f, x), atol=1e-7)  # differences: 1e-10 + third derivatives
    np.testing.assert_allclose(dw, numeric(f, w), atol=1e-7)


# --- refusals ------------------------------------------------------------------

def rope_cfg(**kw):
    d = dict(rows=4, num_q_heads=2, num_k_heads=1, head_dim=16, num_rope_angles=8, max_positions=32,
             q_stride=0, k_stride=0, q_out_stride=0, k_out_stride=0, epsilon=1e-6, dtype=0)
    d.update(kw)
    return m3.QkNormRopeConfig(*[d[f[0]] for f in m3.QkNormRopeConfig._fields_])


def call_rope(lib, cfg, **ptr):
    names = ("q", "k", "wq", "wk", "cos", "sin", "pos", "qo", "ko")
    return lib.m3_qk_norm_rope(ctypes.byref(cfg) if cfg else None,
                               *[ptr.get(n, FAKE) for n in names], None)


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(rows=1 << 31), dict(num_q_heads=-1), dict(num_q_heads=0, num_k_heads=0),
    dict(head_dim=0), dict(head_dim=257), dict(num_rope_angles=9), dict(num_rope_angles=-1),
    dict(max_positions=0), dict(epsilon=0.0), dict(epsilon=float("nan")), dict(dtype=2),
    dict(q_stride=31), dict(k_stride=15), dict(q_out_stride=-1), dict(k_out_stride=1)])
def test_rope_refuses_bad_configs(lib, bad):
    before = m3.launch_count()
    assert call_rope(lib, rope_cfg(**bad)) == m3.M3_ERR_INVALID_ARGUMENT
    assert m3.launch_count() == before


def test_rope_refuses_bad_pointers(lib):
    inv, una = m3.M3_ERR_INVALID_ARGUMENT, m3.M3_ERR_UNALIGNED
    assert call_rope(lib, None) == inv
    for p in ("q", "k", "cos", "sin", "qo", "ko"):
        assert call_rope(lib, rope_cfg(), **{p: None}) == inv, p
    for p in ("wq", "wk", "cos", "sin"):
        assert call_rope(lib, rope_cfg(), **{p: FAKE4}) == una, p
    assert call_rope(lib, rope_cfg(), q=FAKE + 2) == una
    assert call_rope(lib, rope_cfg(rows=40), pos=None) == inv  # more rows than positions
    assert call_rope(lib, rope_cfg(rows=0), q=None, k=None, qo=None, ko=None) == m3.M3_OK


def test_rope_backward_wants_its_workspace(lib):
    cfg = rope_cfg()
    need = m3.m3_qk_norm_rope_backward_workspace(cfg)
    call = lambda ws, n, gw=FAKE: lib.m3_qk_norm_rope_backward(  # noqa: E731
        ctypes.byref(cfg), *[FAKE] * 11, gw, FAKE, ws, n, None)
    assert call(None, need) == m3.M3_ERR_WORKSPACE
    assert call(FAKE, need - 1) == m3.M3_ERR_WORKSPACE
    assert call(FAKE4, need) == m3.M3_ERR_UNALIGNED
    assert call(FAKE, need, FAKE4) == m3.M3_ERR_UNALIGNED


def la_cfg(**kw):
    d = dict(batch_size=2, sequence_length=8, total_rows=16, num_heads=4, num_groups=2, head_dim=16,
             state_size=32, num_slots=0, q_stride=0, k_stride=0, v_stride=0, out_stride=0, scale=1.0,
             dtype=1)
    d.update(kw)
    return m3.LinearAttentionConfig(*[d[f[0]] for f in m3.LinearAttentionConfig._fields_])


BIG = 1 << 40  # a workspace size no call needs more than


def call_fwd(lib, cfg, ws=FAKE, n=BIG, **ptr):
    names = ("q", "k", "v", "ld", "off", "s0", "out", "fin")
    ptr.setdefault("off", None)
    return lib.m3_linear_attention_forward(ctypes.byref(cfg) if cfg else None,
                                           *[ptr.get(x, FAKE) for x in names], ws, n, None)


def call_bwd(lib, cfg, ws=FAKE, n=BIG, **ptr):
    names = ("do", "q", "k", "v", "ld", "off", "s0", "ds", "dq", "dk", "dv", "ds0")
    ptr.setdefault("off", None)
    return lib.m3_linear_attention_backward(ctypes.byref(cfg) if cfg else None,
                                            *[ptr.get(x, FAKE) for x in names], ws, n, None)


def call_step(lib, cfg, **ptr):
    names = ("q", "k", "v", "ld", "slots", "state", "out")
    return lib.m3_linear_attention_step(ctypes.byref(cfg) if cfg else None,
                                        *[ptr.get(x, FAKE) for x in names], None)


@pytest.mark.parametrize("bad", [
    dict(batch_size=0), dict(sequence_length=0), dict(num_heads=0), dict(num_groups=-1),
    dict(num_groups=3), dict(head_dim=0), dict(head_dim=129), dict(state_size=0),
    dict(state_size=129), dict(total_rows=15), dict(total_rows=-1), dict(dtype=7),
    dict(scale=float("inf")), dict(q_stride=63), dict(v_stride=-64), dict(out_stride=63),
    dict(num_slots=-1), dict(batch_size=1 << 40)])
def test_linear_attention_refuses_bad_configs(lib, bad):
    before = m3.launch_count()
    for call in (call_fwd, call_bwd, call_step):
        assert call(lib, la_cfg(**bad)) == m3.M3_ERR_INVALID_ARGUMENT
    assert m3.launch_count() == before


def test_linear_attention_refuses_bad_pointers(lib):
    inv, una, wsp = m3.M3_ERR_INVALID_ARGUMENT, m3.M3_ERR_UNALIGNED, m3.M3_ERR_WORKSPACE
    for call, names in ((call_fwd, ("q", "k", "v", "ld", "out")),
                        (call_bwd, ("do", "q", "k", "v", "ld", "dq", "dk", "dv"))):
        assert call(lib, None) == inv
        for p in names:
            assert call(lib, la_cfg(), **{p: None}) == inv, p
            assert call(lib, la_cfg(), **{p: FAKE + 1}) == una, p
        assert call(lib, la_cfg(), s0=FAKE4) == una
        assert call(lib, la_cfg(), off=FAKE + 2) == una
        assert call(lib, la_cfg(), ws=None) == wsp
        assert call(lib, la_cfg(), n=8) == wsp
        assert call(lib, la_cfg(), ws=FAKE4) == una
    assert call_fwd(lib, la_cfg(), fin=FAKE4) == una
    assert call_bwd(lib, la_cfg(), ds=FAKE4) == una
    assert call_bwd(lib, la_cfg(), ds0=FAKE4) == una


def test_step_refusals(lib):
    one = dict(sequence_length=1, total_rows=2)
    inv = m3.M3_ERR_INVALID_ARGUMENT
    assert call_step(lib, la_cfg(num_slots=4)) == inv              # a sequence is one token
    assert call_step(lib, la_cfg(**one), slots=FAKE) == inv        # slots without a pool
    assert call_step(lib, la_cfg(**one, num_slots=1), slots=None) == inv
    for p in ("q", "k", "v", "ld", "state", "out"):
        assert call_step(lib, la_cfg(**one, num_slots=4), **{p: None}) == inv, p
    assert call_step(lib, la_cfg(**one, num_slots=4), state=FAKE4) == m3.M3_ERR_UNALIGNED
    assert call_step(lib, la_cfg(**one, num_slots=4), slots=FAKE + 1) == m3.M3_ERR_UNALIGNED


def test_binding_refuses_other_tensors():
    import torch
    q = torch.zeros(4, 2, 8)
    with pytest.raises(TypeError):
        m3.qk_norm_rope_config(q.half(), None, num_rope_angles=0)
    with pytest.raises(TypeError):
        m3.qk_norm_rope_config(q.transpose(1, 2), None, num_rope_angles=0)
    with pytest.raises(TypeError):  # rows that are not evenly spaced
        m3.qk_norm_rope_config(torch.zeros(4, 6, 2, 8)[:, ::2][:, :2], torch.zeros(3, 2, 2, 8)[:, :1],
                               num_rope_angles=0)
        m3.qk_norm_rope_config(torch.zeros(3, 5, 2, 8)[:, :4], None, num_rope_angles=0)
    cfg = m3.qk_norm_rope_config(q, None, num_rope_angles=0)
    with pytest.raises(TypeError):  # not on the GPU
        m3.m3_qk_norm_rope(cfg, q, None, None, None, None, None, None, q, None)
    packed = torch.zeros(6, 40)
    view = packed[:, 8:24].view(6, 2, 8)
    assert m3.qk_norm_rope_config(view, None, num_rope_angles=0).q_stride == 40


def test_autograd_refuses_a_gradient_of_the_decays():
    import torch
    from selective_state_space_mamba3_gb300 import autograd
    x = torch.zeros(4, 1, 8)
    with pytest.raises(ValueError):
        autograd.linear_attention(x, x, x, torch.zeros(1, requires_grad=True), 1, 4)

"""Linear-attention operators on the GPU against their plain float64
statements (tests/linattn_ref.py, which also derives the tolerances)."""
import numpy as np
import pytest

import linattn_ref as ref
import selective_state_space_mamba3_gb300 as m3

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from selective_state_space_mamba3_gb300 import build
    build.build()


def torch_dtype(name):
    import torch
    return {"fp32": torch.float32, "bf16": torch.bfloat16}[name]


def bar(dtype):
    return ref.F32_BAR if dtype == "fp32" else ref.BF16_BAR


def dev(a, dtype="fp32"):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(torch_dtype(dtype))


def host(t):
    return t.double().cpu().numpy()


def ws_of(n):
    import torch
    return torch.full((max(n, 16),), 255, dtype=torch.uint8, device="cuda")


def unit(x):
    return x / np.sqrt((x ** 2).mean(-1, keepdims=True) + 1e-6)


class Problem:
    """Inputs of one call, rounded to the activations' type, on both sides."""

    def __init__(self, B, L, H, G, P, N, dtype, lens=None, states=False, seed=0, decay=None):
        import torch
        rng = np.random.default_rng(seed)
        self.B, self.L, self.H, self.G, self.P, self.N, self.dtype = B, L, H, G or H, P, N, dtype
        self.offsets = None if lens is None else np.concatenate([[0], np.cumsum(lens)])
        rows = B * L if lens is None else int(self.offsets[-1])
        self.rows = rows
        t = {}
        t["q"], t["k"] = (unit(rng.standard_normal((rows, self.G, N))) for _ in range(2))
        t["v"], t["do"] = rng.standard_normal((rows, H, P)), rng.standard_normal((rows, H, P))
        self.d = {x: dev(a, dtype) for x, a in t.items()}
        self.h = {x: host(a) for x, a in self.d.items()}
        ld = -(2.0 ** -np.linspace(0.5, 8, H)) if decay is None else np.full(H, decay)
        self.ld = dev(ld)
        self.ld_h = host(self.ld)
        self.s0 = self.ds = None
        if states:
            self.s0, self.ds = dev(rng.standard_normal((B, H, P, N))), dev(
                rng.standard_normal((B, H, P, N)))
        self.scale = 1 / np.sqrt(N)
        self.off_d = None if lens is None else torch.tensor(self.offsets, dtype=torch.int32).cuda()
        groups = 0 if self.G == H else self.G
        self.cfg = m3.linear_attention_config(
            self.d["q"], self.d["k"], self.d["v"], batch_size=B, sequence_length=L, num_heads=H,
            num_groups=groups, scale=self.scale)
        self.scale = self.cfg.scale  # as float32

    def states_h(self):
        return [None if t is None else host(t) for t in (self.s0, self.ds)]

    def forward(self, final=True):
        import torch
        out = torch.full((self.rows, self.H, self.P), float("nan"), device="cuda",
                         dtype=torch_dtype(self.dtype))
        fin = torch.full((self.B, self.H, self.P, self.N), float("nan"), device="cuda")
        ws = ws_of(m3.m3_linear_attention_forward_workspace(self.cfg))
        m3.m3_linear_attention_forward(self.cfg, self.d["q"], self.d["k"], self.d["v"], self.ld,
                                       self.off_d, self.s0, out, fin if final else None, ws)
        assert m3.m3_workspace_status(ws) == m3.M3_OK
        return out, fin

    def backward(self):
        import torch
        grads = [torch.full_like(self.d[x], float("nan")) for x in "qkv"]
        g0 = torch.full((self.B, self.H, self.P, self.N), float("nan"), device="cuda")
        ws = ws_of(m3.m3_linear_attention_backward_workspace(self.cfg))
        m3.m3_linear_attention_backward(self.cfg, self.d["do"], self.d["q"], self.d["k"],
                                        self.d["v"], self.ld, self.off_d, self.s0, self.ds, *grads,
                                        g0, ws)
        assert m3.m3_workspace_status(ws) == m3.M3_OK
        return grads + [g0]

    def ref_forward(self):
        return ref.forward(self.h["q"], self.h["k"], self.h["v"], self.ld_h, self.scale, self.B,
                           self.L, self.offsets, self.states_h()[0])

    def ref_backward(self):
        return ref.backward(self.h["do"], self.h["q"], self.h["k"], self.h["v"], self.ld_h,
                            self.scale, self.B, self.L, self.offsets, *self.states_h())

    def check(self, backward=True):
        (out, fin), (ro, rf) = self.forward(), self.ref_forward()
        errs = {"out": (ref.rel(host(out), ro), bar(self.dtype)),
                "final": (ref.rel(host(fin), rf), ref.F32_BAR)}
        if backward:
            got, want = self.backward(), self.ref_backward()
            for name, a, b in zip(("dq", "dk", "dv", "ds0"), got, want):
                errs[name] = (ref.rel(host(a), b), ref.F32_BAR if name == "ds0" else bar(self.dtype))
        assert all(e <= t for e, t in errs.values()), errs


DTYPES = ["fp32", "bf16"]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("L", [1, 2, 16, 17, 31, 32, 33, 127, 128, 129, 300])
def test_lengths(dtype, L):
    Problem(2, L, 3, 0, 64, 128, dtype, states=L % 2 == 1, seed=L).check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("P,N", [(64, 64), (128, 128), (128, 64), (16, 32), (80, 96), (37, 53), (1, 1),
                                 (8, 120), (72, 8), (127, 128), (100, 4)])
def test_widths(dtype, P, N):
    Problem(2, 150, 2, 0, P, N, dtype, states=True, seed=P * 200 + N).check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("P,N,lens", [(128, 96, [12, 0, 3]), (37, 53, [1, 16]), (1, 1, [2]),
                                      (64, 128, [16] * 200)])
def test_short_sequences(dtype, P, N, lens):
    Problem(len(lens), 16, 4, 2, P, N, dtype, lens=lens, states=True, seed=P).check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H,G", [(6, 1), (6, 2), (4, 4), (1, 1)])
def test_shared_queries_and_keys(dtype, H, G):
    Problem(2, 140, H, G, 64, 128, dtype, states=True, seed=H * 10 + G).check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("G", [0, 1])
@pytest.mark.parametrize("lens", [[5, 0, 129, 1, 128, 300], [0, 0, 0], [1, 1, 1], [257]])
def test_ragged_batches(dtype, G, lens):
    p = Problem(len(lens), max(max(lens), 1), 4, G, 64, 64, dtype, lens=lens, states=True, seed=3)
    p.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", [None, [2100, 0, 700]])
def test_long_sequences_are_cut_into_segments(dtype, lens):
    B = 1 if lens is None else len(lens)
    Problem(B, 2100, 2, 0, 64, 128, dtype, lens=lens, states=True, seed=4).check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("decay", [0.0, -1e-4, -0.5, -0.51, -3.0, -80.0, -200.0, 0.01])
def test_decays(dtype, decay):
    Problem(1, 200, 2, 0, 64, 64, dtype, states=True, seed=6, decay=decay).check()


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_decay_of_minus_infinity_keeps_the_token_alone(dtype):
    p = Problem(1, 150, 2, 0, 64, 64, dtype, states=True, seed=7, decay=-np.inf)
    out, fin = p.forward()
    k, v, q = p.h["k"], p.h["v"], p.h["q"]
    want = p.scale * (q * k).sum(-1, keepdims=True) * v
    assert ref.rel(host(out), want) <= bar(dtype)
    assert ref.rel(host(fin)[0], v[-1][:, :, None] * k[-1][:, None, :]) <= ref.F32_BAR


@pytest.mark.parametrize("dtype", DTYPES)
def test_strided_operands_in_packed_rows(dtype):
    import torch
    p = Problem(2, 140, 2, 0, 64, 128, dtype, seed=8)
    for pad in (0, 8, 3):  # a stride that tile copies take, and one that they do not
        w = 2 * 128 + 2 * 128 + 2 * 64 + pad
        packed = torch.full((p.rows, w), float("nan"), device="cuda", dtype=torch_dtype(dtype))
        views = []
        at = pad
        for x, n in (("q", 256), ("k", 256), ("v", 128)):
            view = packed[:, at:at + n].view(p.rows, *p.d[x].shape[1:])
            view.copy_(p.d[x])
            views.append(view)
            at += n
        out_rows = torch.full((p.rows, 128 + pad), 7.0, device="cuda", dtype=torch_dtype(dtype))
        out = out_rows[:, pad:].view(p.rows, 2, 64)
        cfg = m3.linear_attention_config(*views, batch_size=2, sequence_length=140, scale=p.scale,
                                         out=out)
        ws = ws_of(m3.m3_linear_attention_forward_workspace(cfg))
        m3.m3_linear_attention_forward(cfg, *views, p.ld, None, None, out, None, ws)
        assert ref.rel(host(out), p.ref_forward()[0]) <= bar(dtype)
        assert bool((out_rows[:, :pad] == 7.0).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_of_no_sequence_and_other_sequences_stay_apart(dtype):
    """Rows before the first offset and after the last keep their contents, and
    NaN in one sequence (or in rows of none) reaches no other."""
    import torch
    p = Problem(3, 140, 2, 1, 64, 64, dtype, lens=[50, 140, 90], seed=9)
    pad = lambda t, fill: torch.cat([torch.full_like(t[:3], fill), t, torch.full_like(t[:5], fill)])  # noqa: E731
    d = {x: pad(t, float("nan")) for x, t in p.d.items()}
    lo, hi = 3 + 50, 3 + 190
    d["v"][lo:hi] = float("nan")
    d["k"][lo:hi] = float("inf")
    d["do"][lo:hi] = float("nan")
    off = p.off_d + 3
    cfg = m3.linear_attention_config(d["q"], d["k"], d["v"], batch_size=3, sequence_length=140,
                                     num_heads=2, num_groups=1, scale=p.scale)
    out = torch.full_like(d["v"], 7.0)
    ws = ws_of(m3.m3_linear_attention_forward_workspace(cfg))
    m3.m3_linear_attention_forward(cfg, d["q"], d["k"], d["v"], p.ld, off, None, out, None, ws)
    want = p.ref_forward()[0]
    got = host(out)
    assert (got[:3] == 7).all() and (got[-5:] == 7).all()
    keep = np.r_[0:50, 190:280]
    assert ref.rel(got[3:-5][keep], want[keep]) <= bar(dtype)
    grads = [torch.full_like(d[x], 7.0) for x in "qkv"]
    ws = ws_of(m3.m3_linear_attention_backward_workspace(cfg))
    m3.m3_linear_attention_backward(cfg, d["do"], d["q"], d["k"], d["v"], p.ld, off, None, None,
                                    *grads, None, ws)
    for g, want in zip(grads, p.ref_backward()):
        g = host(g)
        assert (g[:3] == 7).all() and (g[-5:] == 7).all()
        assert ref.rel(g[3:-5][keep], want[keep]) <= bar(dtype)


def test_offsets_outside_the_rows_read_and_write_nothing_outside():
    import torch
    p = Problem(2, 40, 2, 0, 64, 64, "bf16", lens=[40, 30], seed=10)
    good = p.forward()[0]
    p.off_d = torch.tensor([-9, 40, 1000], dtype=torch.int32).cuda()  # taken as 0, 40, 70
    assert torch.equal(p.forward()[0], good)


@pytest.mark.parametrize("dtype", DTYPES)
def test_state_hand_over_in_place(dtype):
    """A sequence in two pieces, the state carried in one buffer, is the whole sequence."""
    import torch
    p = Problem(1, 333, 2, 0, 64, 128, dtype, states=True, seed=11)
    want, fin = p.ref_forward()
    st = p.s0.clone()
    outs = []
    for lo, hi in ((0, 200), (200, 333)):
        q, k, v = (p.d[x][lo:hi].contiguous() for x in "qkv")
        cfg = m3.linear_attention_config(q, k, v, batch_size=1, sequence_length=hi - lo,
                                         scale=p.scale)
        out = torch.empty_like(v)
        ws = ws_of(m3.m3_linear_attention_forward_workspace(cfg))
        m3.m3_linear_attention_forward(cfg, q, k, v, p.ld, None, st, out, st, ws)
        outs.append(out)
    assert ref.rel(host(torch.cat(outs)), want) <= bar(dtype)
    assert ref.rel(host(st), fin) <= ref.F32_BAR


@pytest.mark.parametrize("dtype", DTYPES)
def test_the_same_call_gives_the_same_bits(dtype):
    import torch
    p = Problem(2, 700, 4, 2, 64, 128, dtype, states=True, seed=12)
    a, b = p.forward(), p.forward()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    a, b = p.backward(), p.backward()
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_on_a_stream_of_its_own():
    import torch
    p = Problem(2, 300, 2, 0, 64, 128, "bf16", seed=13)
    want = p.forward()[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = p.forward()[0]
    s.synchronize()
    assert torch.equal(got, want)


def test_gradients_against_differences_of_the_forward_call():
    """A directional derivative of loss = sum(out * do) + sum(final * ds), float32. The loss
    is multilinear, so central differences in one operand have no truncation error; with a
    step as large as the operand their rounding is that of the sums, about 1e-6 of them."""
    import torch
    p = Problem(2, 200, 4, 2, 64, 64, "fp32", states=True, seed=14)
    grads = p.backward()

    def loss():
        out, fin = p.forward()
        return (out.double() * p.d["do"].double()).sum() + (fin.double() * p.ds.double()).sum()

    for x, g in zip(("q", "k", "v", "s0"), grads):
        t = p.s0 if x == "s0" else p.d[x]
        step = torch.randn_like(t)
        old = t.clone()
        t.copy_(old + step)
        hi, step_hi = loss(), t.double() - old.double()
        t.copy_(old - step)
        lo, step_lo = loss(), old.double() - t.double()
        t.copy_(old)
        want = (g.double() * (step_hi + step_lo)).sum()
        size = (g.double().square().sum() * step.double().square().sum()).sqrt()
        assert abs(hi - lo - want) <= 1e-4 * size, x


# --- single tokens ------------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,H,G,P,N", [(1, 4, 0, 64, 128), (5, 6, 2, 64, 64), (3, 2, 1, 37, 53),
                                       (2, 1, 0, 1, 1), (2, 2, 0, 128, 100), (4, 3, 0, 16, 6),
                                       (300, 8, 1, 64, 128)])
def test_step(dtype, B, H, G, P, N):
    import torch
    rng = np.random.default_rng(B * 1000 + P)
    g = G or H
    slots_n = B + 3
    q, k, v = (dev(rng.standard_normal((B, x, w)), dtype) for x, w in ((g, N), (g, N), (H, P)))
    state = dev(rng.standard_normal((slots_n, H, P, N)))
    before = host(state)
    ld = dev(-rng.uniform(0.01, 1, H))
    order = rng.permutation(slots_n)[:B].astype(np.int32)
    dead = [] if B < 4 else [1, 2]
    if dead:
        order[1], order[2] = -1, slots_n  # both outside the pool
    slots = torch.from_numpy(order).cuda()
    out = torch.full((B, H, P), float("nan"), device="cuda", dtype=torch_dtype(dtype))
    cfg = m3.linear_attention_config(q, k, v, batch_size=B, sequence_length=1, num_heads=H,
                                     num_groups=G, scale=0.3, num_slots=slots_n)
    m3.m3_linear_attention_step(cfg, q, k, v, ld, slots, state, out)
    want, fin = before.copy(), np.zeros((B, H, P))
    for b in range(B):
        if b in dead:
            continue
        o, s = ref.forward(host(q)[b:b + 1], host(k)[b:b + 1], host(v)[b:b + 1], host(ld), cfg.scale,
                           1, 1, None, before[order[b]][None])
        want[order[b]], fin[b] = s[0], o[0]
    assert ref.rel(host(state), want) <= ref.F32_BAR
    idle = np.setdiff1d(np.arange(slots_n), order)
    assert np.array_equal(host(state)[idle], before[idle])
    assert ref.rel(host(out), fin) <= (ref.F32_BAR if dtype == "fp32" else ref.BF16_ROUND)
    assert all((host(out)[b] == 0).all() for b in dead)


def test_steps_continue_a_prompt():
    import torch
    p = Problem(2, 40, 4, 0, 64, 128, "bf16", seed=15)
    want, fin = p.ref_forward()
    cut = 33
    x = {n: t.view(2, 40, *t.shape[1:]) for n, t in p.d.items()}
    q, k, v = (x[n][:, :cut] for n in "qkv")
    q, k, v = (t.reshape(2 * cut, *t.shape[2:]) for t in (q, k, v))
    cfg = m3.linear_attention_config(q, k, v, batch_size=2, sequence_length=cut, scale=p.scale)
    st = torch.empty(2, 4, 64, 128, device="cuda")
    out = torch.empty(2, 40, 4, 64, device="cuda", dtype=torch.bfloat16)
    first = torch.empty_like(v)
    ws = ws_of(m3.m3_linear_attention_forward_workspace(cfg))
    m3.m3_linear_attention_forward(cfg, q, k, v, p.ld, None, None, first, st, ws)
    out[:, :cut] = first.view(2, cut, 4, 64)
    for t in range(cut, 40):
        q, k, v = (x[n][:, t].contiguous() for n in "qkv")
        cfg = m3.linear_attention_config(q, k, v, batch_size=2, sequence_length=1, scale=p.scale)
        one = torch.empty_like(v)
        m3.m3_linear_attention_step(cfg, q, k, v, p.ld, None, st, one)
        out[:, t] = one
    assert ref.rel(host(out).reshape(80, 4, 64), want) <= ref.BF16_BAR
    assert ref.rel(host(st), fin) <= ref.F32_BAR


# --- norm and rotation ----------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,hq,hk,D,A,packed", [
    (1, 1, 1, 64, 32, False), (5, 4, 1, 128, 64, True), (7, 3, 3, 128, 32, True),
    (300, 8, 2, 80, 40, False), (9, 2, 0, 96, 24, False), (4, 0, 5, 256, 128, True),
    (6, 2, 2, 64, 0, False), (11, 3, 2, 37, 11, False), (3, 2, 1, 200, 100, True),
    (2000, 9, 4, 64, 32, True), (3, 1, 2, 1, 0, False), (13, 2, 2, 248, 7, True)])
def test_norm_and_rotation(dtype, rows, hq, hk, D, A, packed):
    import torch
    rng = np.random.default_rng(rows * 7 + D)
    td = torch_dtype(dtype)
    heads = {"q": hq, "k": hk}
    x, dy, w = {}, {}, {}
    row_w = (hq + hk) * D + (8 if packed else 0)
    buf = torch.full((rows, row_w), float("nan"), device="cuda", dtype=td)
    at = 0
    for n, h in heads.items():
        if not h:
            x[n] = dy[n] = w[n] = None
            continue
        val = dev(rng.standard_normal((rows, h, D)) * 3, dtype)
        x[n] = val
        if packed:
            x[n] = buf[:, at:at + h * D].view(rows, h, D)
            x[n].copy_(val)
            at += h * D
        dy[n] = dev(rng.standard_normal((rows, h, D)), dtype)
        w[n] = dev(rng.uniform(0.5, 1.5, D)) if n == "q" else None
    ang = rng.uniform(0, 6.28, (50, A))
    cos, sin = (dev(np.cos(ang)), dev(np.sin(ang))) if A else (None, None)
    posn = rng.integers(0, 50, rows).astype(np.int32)
    if rows > 3:
        posn[1], posn[2] = -1, 50  # not rotated
    pos = torch.from_numpy(posn).cuda() if A else None
    cfg = m3.qk_norm_rope_config(x["q"], x["k"], num_rope_angles=A, max_positions=50, epsilon=1e-5)
    new = lambda n: None if x[n] is None else torch.full((rows, heads[n], D), float("nan"),  # noqa: E731
                                                          device="cuda", dtype=td)
    y = {n: new(n) for n in heads}
    m3.m3_qk_norm_rope(cfg, x["q"], x["k"], w["q"], w["k"], cos, sin, pos, y["q"], y["k"])
    dx, gw = {n: new(n) for n in heads}, {n: torch.full((D,), float("nan"), device="cuda")
                                          if heads[n] else None for n in heads}
    ws = ws_of(m3.m3_qk_norm_rope_backward_workspace(cfg))
    m3.m3_qk_norm_rope_backward(cfg, x["q"], x["k"], w["q"], w["k"], cos, sin, pos, dy["q"],
                                dy["k"], dx["q"], dx["k"], gw["q"], gw["k"], ws)
    tabs = (None, None) if not A else (host(cos), host(sin))
    # bfloat16: one rounding at the output
    tol = ref.F32_BAR if dtype == "fp32" else ref.BF16_ROUND
    for n in heads:
        if x[n] is None:
            continue
        wn = None if w[n] is None else host(w[n])
        want = ref.rope(host(x[n]), wn, *tabs, posn, cfg.epsilon)
        assert ref.rel(host(y[n]), want) <= tol
        gx, gwn = ref.rope_backward(host(x[n]), wn, *tabs, posn, cfg.epsilon, host(dy[n]))
        if D > 1:  # of one value the norm keeps the sign alone: its gradient vanishes but for epsilon
            assert ref.rel(host(dx[n]), gx) <= tol
        assert ref.rel(host(gw[n]), gwn) <= ref.F32_BAR
    # in place on the packed rows
    m3_cfg = m3.qk_norm_rope_config(x["q"], x["k"], num_rope_angles=A, max_positions=50, epsilon=1e-5,
                                    q_out=x["q"], k_out=x["k"])
    m3.m3_qk_norm_rope(m3_cfg, x["q"], x["k"], w["q"], w["k"], cos, sin, pos, x["q"], x["k"])
    for n in heads:
        if x[n] is not None:
            assert torch.equal(x[n], y[n])


def test_rows_of_zeros_and_their_gradient_are_finite():
    import torch
    x = torch.zeros(2, 1, 64, device="cuda")
    cfg = m3.qk_norm_rope_config(x, None, num_rope_angles=0, epsilon=1e-6)
    y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(64, device="cuda")
    m3.m3_qk_norm_rope(cfg, x, None, None, None, None, None, None, y, None)
    assert bool((y == 0).all())
    ws = ws_of(m3.m3_qk_norm_rope_backward_workspace(cfg))
    dy = torch.ones_like(x)
    m3.m3_qk_norm_rope_backward(cfg, x, None, None, None, None, None, None, dy, None, dx, None, dw,
                                None, ws)
    assert ref.rel(host(dx), np.full((2, 1, 64), 1e3)) <= ref.F32_BAR
    assert bool((dw == 0).all())


def test_weight_gradients_keep_their_bits():
    import torch
    x, dy = (torch.randn(4000, 8, 128, device="cuda") for _ in range(2))
    cfg = m3.qk_norm_rope_config(x, None, num_rope_angles=0)
    ws = ws_of(m3.m3_qk_norm_rope_backward_workspace(cfg))
    got = []
    for _ in range(2):
        dx, dw = torch.empty_like(x), torch.empty(128, device="cuda")
        m3.m3_qk_norm_rope_backward(cfg, x, None, None, None, None, None, None, dy, None, dx, None,
                                    dw, None, ws)
        got.append(dw)
    assert torch.equal(*got)


# --- as a layer ---------------------------------------------------------------------

def test_autograd_of_a_layer():
    """Packed projection -> norm and rotation -> ragged linear attention, differentiated
    through the bindings, against the composed float64 formulas."""
    import torch
    from selective_state_space_mamba3_gb300 import autograd
    rng = np.random.default_rng(21)
    H, P, N, A, lens = 3, 32, 64, 16, [70, 0, 130]
    rows = sum(lens)
    off = np.concatenate([[0], np.cumsum(lens)])
    proj = dev(rng.standard_normal((rows, H * (2 * N + P)))).requires_grad_()
    wq, wk = (dev(rng.uniform(0.5, 1.5, N)).requires_grad_() for _ in range(2))
    ang = rng.uniform(0, 6.28, (200, A))
    cos, sin = dev(np.cos(ang)), dev(np.sin(ang))
    posn = np.concatenate([np.arange(n) for n in lens]).astype(np.int32)
    s0 = dev(rng.standard_normal((3, H, P, N))).requires_grad_()
    ld = dev(-rng.uniform(0.01, 0.5, H))
    q, k = proj[:, :H * N].view(rows, H, N), proj[:, H * N:2 * H * N].view(rows, H, N)
    v = proj[:, 2 * H * N:].view(rows, H, P)
    qn, kn = autograd.qk_norm_rope(q, k, wq, wk, cos, sin, torch.from_numpy(posn).cuda(), A)
    out, fin = autograd.linear_attention(
        qn, kn, v, ld, 3, 130, scale=0.125, offsets=torch.from_numpy(off.astype(np.int32)).cuda(),
        initial_state=s0, return_state=True)
    do, ds = dev(rng.standard_normal(out.shape)), dev(rng.standard_normal(fin.shape))
    ((out * do).sum() + (fin * ds).sum()).backward()
    hq, hk, hv = host(q.detach()), host(k.detach()), host(v.detach())
    tabs = host(cos), host(sin)
    yq = ref.rope(hq, host(wq.detach()), *tabs, posn, 1e-6)
    yk = ref.rope(hk, host(wk.detach()), *tabs, posn, 1e-6)
    want, want_fin = ref.forward(yq, yk, hv, host(ld), 0.125, 3, 130, off, host(s0.detach()))
    assert ref.rel(host(out.detach()), want) <= ref.F32_BAR
    assert ref.rel(host(fin.detach()), want_fin) <= ref.F32_BAR
    dq, dk, dv, d0 = ref.backward(host(do), yq, yk, hv, host(ld), 0.125, 3, 130, off,
                                  host(s0.detach()), host(ds))
    gq, gwq = ref.rope_backward(hq, host(wq.detach()), *tabs, posn, 1e-6, dq)
    gk, gwk = ref.rope_backward(hk, host(wk.detach()), *tabs, posn, 1e-6, dk)
    want = np.concatenate([x.reshape(rows, -1) for x in (gq, gk, dv)], 1)
    # two operators in a row: twice the bar
    for got, w in ((proj.grad, want), (wq.grad, gwq), (wk.grad, gwk), (s0.grad, d0)):
        assert ref.rel(host(got), w) <= 2 * ref.F32_BAR


def test_calls_captured_into_a_graph_replay_to_the_same_bits():
    import torch
    p = Problem(2, 300, 4, 0, 64, 128, "bf16", states=True, seed=22)
    out = torch.empty_like(p.d["v"])
    fin = torch.empty_like(p.s0)
    ws = ws_of(m3.m3_linear_attention_forward_workspace(p.cfg))
    call = lambda: m3.m3_linear_attention_forward(  # noqa: E731
        p.cfg, p.d["q"], p.d["k"], p.d["v"], p.ld, None, p.s0, out, fin, ws)
    call()
    torch.cuda.synchronize()
    want, want_fin = out.clone(), fin.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    out.zero_(), fin.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(fin, want_fin)


@pytest.mark.parametrize("dtype", DTYPES)
def test_adjoints_captured_into_a_graph_replay_to_the_same_bits(dtype):
    """The three roles run beside each other by programmatic launches, which a graph keeps."""
    import torch
    p = Problem(1, 2100, 4, 2, 64, 128, dtype, states=True, seed=23)  # cut into segments
    want = p.backward()
    grads = [torch.empty_like(p.d[x]) for x in "qkv"]
    g0 = torch.empty_like(p.s0)
    ws = ws_of(m3.m3_linear_attention_backward_workspace(p.cfg))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m3.m3_linear_attention_backward(p.cfg, p.d["do"], p.d["q"], p.d["k"], p.d["v"], p.ld, None,
                                        p.s0, p.ds, *grads, g0, ws)
    for _ in range(2):
        for t in (*grads, g0):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*grads, g0), want))


def test_the_example_runs():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "linear_attention_layer.py")
    spec = importlib.util.spec_from_file_location("linear_attention_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    worst, losses = mod.main()
    assert worst <= ref.BF16_BAR  # steps against the prompt call, on the same inputs
    assert losses[-1] < losses[0]

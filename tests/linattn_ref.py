"""Plain float64 statements of the linear-attention operators, token by token
(numpy, no code shared with the library): the recurrence
S_t = lam S_{t-1} + v_t k_t^T, out_t = scale S_t q_t and its adjoint, and the
norm with rotation and its adjoint.

Tolerances, derived from the arithmetic before any run (relative l2 norms):
- float32: the library's FP32 bar, 1e-5. The longest chains here are under
  600 roundings of 2^-24 with random signs, about 1.5e-6.
- one rounding to bfloat16: its unit roundoff, 2^-8 (8 significant bits).
- bfloat16 outputs of the chunked products: three roundings to bfloat16 lie
  between exact operands and an output (a masked score, a state element, the
  output). Over many values the rms of a rounding is 2^-8 / sqrt(3) times the
  rms of 1 / mantissa, 0.71: 1.6e-3, below 2^-9; three of them: 3 * 2^-9.
- float32 states out of bfloat16 operands: the decayed operand is carried as
  two bfloat16 parts (a relative 2^-18), summed in float32: the FP32 bar.
"""
import numpy as np

F32_BAR = 1e-5
BF16_ROUND = 2.0 ** -8
BF16_BAR = 3 * 2.0 ** -9


def rel(got, ref):
    # every output is float32 or narrower: what float32 cannot hold is not expected
    got, ref = np.asarray(got, np.float64), np.asarray(ref).astype(np.float32).astype(np.float64)
    assert got.shape == ref.shape, (got.shape, ref.shape)
    assert np.array_equal(np.isfinite(got), np.isfinite(ref))
    n = np.linalg.norm(ref)
    d = np.linalg.norm(got - ref)
    return d / n if n else d


def spans(rows, batch, length, offsets):
    if offsets is None:
        return [(b * length, (b + 1) * length) for b in range(batch)]
    return [(int(a), int(z)) for a, z in zip(offsets[:-1], offsets[1:])]


def forward(q, k, v, log_decay, scale, batch, length, offsets=None, initial=None):
    """q, k [rows, G, N], v [rows, H, P] -> out [rows, H, P], final [B, H, P, N]."""
    H, P, N = v.shape[1], v.shape[2], q.shape[2]
    rep = H // q.shape[1]
    q, k = np.repeat(q, rep, 1), np.repeat(k, rep, 1)
    with np.errstate(over="ignore"):
        lam = np.exp(np.asarray(log_decay, np.float64))[:, None, None]
    out = np.zeros(v.shape)
    final = np.zeros((batch, H, P, N)) if initial is None else np.array(initial, np.float64)
    for b, (lo, hi) in enumerate(spans(len(q), batch, length, offsets)):
        S = final[b]
        for t in range(lo, hi):
            S = lam * S + v[t][:, :, None] * k[t][:, None, :]
            out[t] = scale * np.einsum("hpn,hn->hp", S, q[t])
        final[b] = S
    return out, final


def backward(do, q, k, v, log_decay, scale, batch, length, offsets=None, initial=None, dfinal=None):
    H, P, N, G = v.shape[1], v.shape[2], q.shape[2], q.shape[1]
    rep = H // G
    q, k = np.repeat(q, rep, 1), np.repeat(k, rep, 1)
    lam = np.exp(np.asarray(log_decay, np.float64))[:, None, None]
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    dinit = np.zeros((batch, H, P, N))
    for b, (lo, hi) in enumerate(spans(len(q), batch, length, offsets)):
        S = np.zeros((H, P, N)) if initial is None else np.array(initial[b], np.float64)
        for t in range(lo, hi):
            S = lam * S + v[t][:, :, None] * k[t][:, None, :]
            dq[t] = scale * np.einsum("hpn,hp->hn", S, do[t])
        R = np.zeros((H, P, N)) if dfinal is None else np.array(dfinal[b], np.float64)
        for t in range(hi - 1, lo - 1, -1):
            R = R + scale * do[t][:, :, None] * q[t][:, None, :]
            dk[t] = np.einsum("hpn,hp->hn", R, v[t])
            dv[t] = np.einsum("hpn,hn->hp", R, k[t])
            R = lam * R
        dinit[b] = R
    fold = lambda x: x.reshape(len(x), G, rep, N).sum(2)  # noqa: E731
    return fold(dq), fold(dk), dv, dinit


def rope(x, w, cos, sin, pos, eps):
    """x [rows, heads, D] -> y; cos, sin [positions, A], pos [rows] (outside: not rotated)."""
    D, A = x.shape[-1], 0 if cos is None else cos.shape[1]
    u = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    if w is not None:
        u = u * w
    y = u.copy()
    for r in range(len(x)):
        if A and 0 <= pos[r] < len(cos):
            c, s = cos[pos[r]].astype(np.float64), sin[pos[r]].astype(np.float64)
            y[r, :, :A] = u[r, :, :A] * c - u[r, :, A:2 * A] * s
            y[r, :, A:2 * A] = u[r, :, :A] * s + u[r, :, A:2 * A] * c
    assert y.shape[-1] == D
    return y


def rope_backward(x, w, cos, sin, pos, eps, dy):
    A = 0 if cos is None else cos.shape[1]
    g = np.array(dy, np.float64)
    for r in range(len(x)):
        if A and 0 <= pos[r] < len(cos):
            c, s = cos[pos[r]].astype(np.float64), sin[pos[r]].astype(np.float64)
            lo, hi = g[r, :, :A].copy(), g[r, :, A:2 * A].copy()
            g[r, :, :A] = lo * c + hi * s
            g[r, :, A:2 * A] = hi * c - lo * s
    inv = 1 / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    xh = x * inv
    dw = (g * xh).sum((0, 1))
    if w is not None:
        g = g * w
    return inv * (g - xh * (g * xh).mean(-1, keepdims=True)), dw

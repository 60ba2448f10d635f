"""torch.autograd bindings of the SISO and MIMO scans: the forward through
m3_siso_forward / m3_mimo_forward and the gradients through m3_siso_backward /
m3_mimo_backward (oarust mamba3.rs `mamba3_siso` / `mamba3_siso_backward` and
`mamba3_mimo` / `mamba3_mimo_backward`: each scan with its adjoint). Argument marshalling only: outputs, gradients and workspaces are
torch allocations on the inputs' device and stream, and every step runs in
libm3's kernels.

    out = siso_scan(cfg, c, b, x, z, adt, dt, trap, angle, c_bias, b_bias, d)
    out = mimo_scan(cfg, c, b, x, z, adt, dt, trap, angle, c_bias, b_bias, d,
                    mimo_x, mimo_z, mimo_o, norm_weight)
    x, z, bh, ch, dt, adt, trap, angle = preprocess(pcfg, projected, dt_bias)

preprocess pairs m3_preprocess with m3_preprocess_backward (`mamba3_preprocess`
/ `mamba3_preprocess_backward`); pcfg is the preprocess config dict of the C
ABI (inner_size, state_size, num_heads, num_rope_angles, num_groups,
mimo_rank, epsilon, dt_min, dt_max, a_floor) and the outputs are 2-D, one row
per packed row.

    q, k = qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions, num_rope_angles)
    out = linear_attention(q, k, v, log_decay, batch_size, sequence_length, ...)

The last two are the layers' own operators (m3_qk_norm_rope,
m3_linear_attention_forward and their adjoints); their activations may be
float32 or bfloat16 and rows of a packed projection. Gradients of the decays and
of the rotation tables are refused, and so are second derivatives.

cfg is the SsmConfig dict of the C ABI (batch_size, sequence_length, num_heads,
num_groups, head_dim, state_size, num_rope_angles, mimo_rank, has_z, has_d,
has_output_norm); math_mode picks the forward's arithmetic (the gradients are
FP32 in either mode). Every tensor must be a contiguous float32 CUDA tensor in
the C ABI's layout; angle may be None when num_rope_angles is 0.
"""
from __future__ import annotations

import torch

from . import _binding as m3

def _workspace(nbytes, like):
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=like.device)


def _grads_like(tensors):
    return [None if t is None else torch.empty_like(t) for t in tensors]


class _SisoScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, cfg, math_mode, *ops):
        c = m3.ssm_config(cfg, math_mode)
        x = ops[2]
        out = torch.empty_like(x)
        ws = _workspace(m3.m3_siso_forward_workspace(c), x)
        m3.m3_siso_forward(c, *ops, out, ws)
        ctx.cfg = cfg
        ctx.save_for_backward(*[t if t is not None else torch.empty(0) for t in ops])
        ctx.angle_none = ops[7] is None
        return out

    @staticmethod
    def backward(ctx, grad_out):
        ops = list(ctx.saved_tensors)
        if ctx.angle_none:
            ops[7] = None
        c = m3.ssm_config(ctx.cfg, m3.M3_MATH_FP32)
        grads = _grads_like(ops)
        ws = _workspace(m3.m3_siso_backward_workspace(c), grad_out)
        m3.m3_siso_backward(c, grad_out.contiguous(), *ops, *grads, ws)
        return (None, None, *grads)


class _MimoScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, cfg, math_mode, *ops):
        c = m3.ssm_config(cfg, math_mode)
        x = ops[2]
        out = torch.empty_like(x)
        ws = _workspace(m3.m3_mimo_forward_workspace(c), x)
        m3.m3_mimo_forward(c, *ops, out, ws)
        ctx.cfg = cfg
        ctx.save_for_backward(*[t if t is not None else torch.empty(0) for t in ops])
        ctx.angle_none = ops[7] is None
        return out

    @staticmethod
    def backward(ctx, grad_out):
        ops = list(ctx.saved_tensors)
        if ctx.angle_none:
            ops[7] = None
        c = m3.ssm_config(ctx.cfg, m3.M3_MATH_FP32)
        grads = _grads_like(ops)
        ws = _workspace(m3.m3_mimo_backward_workspace(c), grad_out)
        m3.m3_mimo_backward(c, grad_out.contiguous(), *ops, *grads, ws)
        return (None, None, *grads)


def _widths(pcfg):
    """Columns of the eight preprocess outputs: x, z, bh, ch, dt, adt, trap, angle."""
    I, H, A = pcfg["inner_size"], pcfg["num_heads"], pcfg["num_rope_angles"]
    bc = pcfg["num_groups"] * pcfg["mimo_rank"] * pcfg["state_size"]
    return (I, I, bc, bc, H, H, H, A)


class _Preprocess(torch.autograd.Function):
    @staticmethod
    def forward(ctx, pcfg, projected, dt_bias):
        c = m3.preprocess_config(**pcfg)
        rows = projected.shape[0]
        outs = [torch.empty(rows, n, device=projected.device) for n in _widths(pcfg)]
        m3.m3_preprocess(c, rows, projected, dt_bias, *outs)
        ctx.pcfg = pcfg
        ctx.save_for_backward(projected, dt_bias)
        return tuple(outs)

    @staticmethod
    def backward(ctx, *grads):
        projected, dt_bias = ctx.saved_tensors
        c = m3.preprocess_config(**ctx.pcfg)
        rows = projected.shape[0]
        # an output the loss does not use contributes a zero gradient
        g = [torch.zeros(rows, n, device=projected.device) if gr is None else gr.contiguous()
             for gr, n in zip(grads, _widths(ctx.pcfg))]
        gp = torch.empty_like(projected)
        gb = torch.empty_like(dt_bias)
        ws = _workspace(m3.m3_preprocess_backward_workspace(c, rows), projected)
        m3.m3_preprocess_backward(c, rows, projected, dt_bias, *g, gp, gb, ws)
        return None, gp, gb


def preprocess(pcfg, projected, dt_bias):
    """`mamba3_preprocess` with its adjoint: (x, z, bh, ch, dt, adt, trap, angle)."""
    return _Preprocess.apply(dict(pcfg), projected, dt_bias)


def siso_scan(cfg, c, b, x, z, adt, dt, trap, angle, c_bias, b_bias, d,
              math_mode=m3.M3_MATH_FP32):
    """`mamba3_siso` with its adjoints: out [B,L,H,P]."""
    return _SisoScan.apply(dict(cfg), math_mode, c, b, x, z, adt, dt, trap, angle, c_bias,
                           b_bias, d)


def mimo_scan(cfg, c, b, x, z, adt, dt, trap, angle, c_bias, b_bias, d, mimo_x, mimo_z, mimo_o,
              norm_weight, math_mode=m3.M3_MATH_FP32):
    """`mamba3_mimo` with its adjoints: out [B,L,H,P]."""
    return _MimoScan.apply(dict(cfg), math_mode, c, b, x, z, adt, dt, trap, angle, c_bias,
                           b_bias, d, mimo_x, mimo_z, mimo_o, norm_weight)


class _NoDerivative(torch.autograd.Function):
    @staticmethod
    def forward(ctx, grad):
        return grad.view_as(grad)

    @staticmethod
    def backward(ctx, grad):
        raise RuntimeError("the adjoints of the linear-attention operators are once_differentiable: "
                           "they have no derivative themselves")


def _once_differentiable(backward):
    """Gradients made with create_graph=True carry a graph that raises. (torch's own mark
    of this name leaves it out where the incoming gradients need none, though the operands'
    gradients depend on the operands all the same.)"""
    def once(ctx, *grads):
        with torch.no_grad():
            out = backward(ctx, *grads)
        if not torch.is_grad_enabled():
            return out
        return tuple(None if g is None else _NoDerivative.apply(g.requires_grad_()) for g in out)
    return once


class _QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, num_rope_angles, max_positions, epsilon, cos, sin, positions, q, k, q_weight,
                k_weight):
        cfg = m3.qk_norm_rope_config(q, k, num_rope_angles=num_rope_angles,
                                     max_positions=max_positions, epsilon=epsilon)
        outs = [None if t is None else torch.empty(t.shape, dtype=t.dtype, device=t.device)
                for t in (q, k)]
        m3.m3_qk_norm_rope(cfg, q, k, q_weight, k_weight, cos, sin, positions, *outs)
        ctx.cfg = cfg
        # the tables too: one that is written again before the backward call is an error
        ctx.save_for_backward(q, k, q_weight, k_weight, cos, sin, positions)
        ctx.set_materialize_grads(False)
        return tuple(outs)

    @staticmethod
    @_once_differentiable
    def backward(ctx, *grads):
        q, k, wq, wk, *tables = ctx.saved_tensors
        some = q if q is not None else k
        dy = [None if t is None else torch.zeros(t.shape, dtype=t.dtype, device=t.device)
              if g is None else g.contiguous() for t, g in zip((q, k), grads)]
        dx = [None if g is None else torch.empty_like(g) for g in dy]
        dw = [None if w is None else torch.empty_like(w) for w in (wq, wk)]
        ws = _workspace(m3.m3_qk_norm_rope_backward_workspace(ctx.cfg), some)
        m3.m3_qk_norm_rope_backward(ctx.cfg, q, k, wq, wk, *tables, *dy, *dx, *dw, ws)
        return (None,) * 6 + (*dx, *dw)


def qk_norm_rope(q, k, q_weight, k_weight, cos_table, sin_table, positions, num_rope_angles,
                 epsilon=1e-6):
    """Norm and rotation of query and key heads (m3_qk_norm_rope) with its adjoint:
    the normalised, rotated q and k, dense. q or k, and each weight, may be None. The
    rotation is fixed: its tables get no gradient."""
    if any(t is not None and t.requires_grad for t in (cos_table, sin_table)):
        raise ValueError("the rotation is fixed: its tables get no gradient")
    rows = 0 if cos_table is None else cos_table.shape[0]
    return _QkNormRope.apply(num_rope_angles, rows, epsilon, cos_table, sin_table, positions, q, k,
                             q_weight, k_weight)


class _LinearAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, batch_size, sequence_length, num_groups, scale, offsets, want_state, log_decay,
                q, k, v, initial_state):
        cfg = m3.linear_attention_config(q, k, v, batch_size=batch_size,
                                         sequence_length=sequence_length, num_groups=num_groups,
                                         scale=scale)
        # rows of no sequence are not written
        new = torch.empty if offsets is None else torch.zeros
        out = new(v.shape, dtype=v.dtype, device=v.device)
        final = None
        if want_state:
            final = torch.empty(batch_size, v.shape[-2], v.shape[-1], q.shape[-1],
                                dtype=torch.float32, device=v.device)
        ws = _workspace(m3.m3_linear_attention_forward_workspace(cfg), v)
        m3.m3_linear_attention_forward(cfg, q, k, v, log_decay, offsets, initial_state, out, final, ws)
        ctx.cfg = cfg
        ctx.save_for_backward(log_decay, offsets, q, k, v, initial_state)
        ctx.set_materialize_grads(False)  # an unused final state is a NULL gradient, not zeros to read
        return out, final

    @staticmethod
    @_once_differentiable
    def backward(ctx, grad_out, grad_final):
        log_decay, offsets, q, k, v, initial = ctx.saved_tensors
        new = torch.empty if offsets is None else torch.zeros
        if grad_out is None:
            grad_out = torch.zeros(v.shape, dtype=v.dtype, device=v.device)
        grads = [new(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v)]
        d_init = None if initial is None else torch.empty_like(initial)
        ws = _workspace(m3.m3_linear_attention_backward_workspace(ctx.cfg), v)
        m3.m3_linear_attention_backward(
            ctx.cfg, grad_out.contiguous(), q, k, v, log_decay, offsets, initial,
            None if grad_final is None else grad_final.contiguous(), *grads, d_init, ws)
        return (None,) * 7 + (*grads, d_init)


def linear_attention(q, k, v, log_decay, batch_size, sequence_length, num_groups=0, scale=1.0,
                     offsets=None, initial_state=None, return_state=False):
    """Causal linear attention with a decay per head (m3_linear_attention_forward) with its
    adjoints: out [..., heads, head_dim], and with return_state the final states too. The
    decays are fixed: log_decay gets no gradient."""
    if log_decay.requires_grad:
        raise ValueError("the decays are fixed: log_decay gets no gradient")
    out, final = _LinearAttention.apply(batch_size, sequence_length, num_groups, scale, offsets,
                                        return_state, log_decay, q, k, v, initial_state)
    return (out, final) if return_state else out

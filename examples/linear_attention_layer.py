"""A linear-attention layer as a hybrid model runs it beside its selective-state layers.

Serving: a ragged batch of prompts goes through one packed projection; queries
and keys are normalised and rotated in place in its rows; linear attention runs
over the prompts and leaves its states in a pool of slots; then every sequence
decodes a few tokens from its slot. The same tokens, run as part of a longer
prompt, give the same outputs.

Training: a few steps of gradient descent through the same operators.

    python examples/linear_attention_layer.py
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_state_space_mamba3_gb300 as m3  # noqa: E402
from selective_state_space_mamba3_gb300 import autograd  # noqa: E402

HEADS, HEAD_DIM, STATE, ANGLES, WIDTH = 8, 64, 128, 32, 256
QK, V = HEADS * STATE, HEADS * HEAD_DIM
SCALE = 1 / math.sqrt(STATE)


def tables(length):
    freq = 10000.0 ** (-torch.arange(ANGLES, device="cuda", dtype=torch.float64) / ANGLES)
    ang = torch.arange(length, device="cuda", dtype=torch.float64)[:, None] * freq
    return ang.cos().float(), ang.sin().float()


def split(proj):
    """Queries, keys and values as views of packed rows."""
    rows = proj.shape[0]
    return (proj[:, :QK].view(rows, HEADS, STATE), proj[:, QK:2 * QK].view(rows, HEADS, STATE),
            proj[:, 2 * QK:].view(rows, HEADS, HEAD_DIM))


def norm_rope_(q, k, weights, tabs, positions):
    cfg = m3.qk_norm_rope_config(q, k, num_rope_angles=ANGLES, max_positions=tabs[0].shape[0],
                                 q_out=q, k_out=k)
    m3.m3_qk_norm_rope(cfg, q, k, *weights, *tabs, positions, q, k)


def prompts(x, w_in, weights, tabs, log_decay, lengths):
    """Rows [sum(lengths), WIDTH] -> outputs and the sequences' final states."""
    q, k, v = split(x @ w_in)
    dev = x.device
    positions = torch.cat([torch.arange(n, dtype=torch.int32, device=dev) for n in lengths])
    norm_rope_(q, k, weights, tabs, positions)
    offsets = torch.tensor([0] + lengths).cumsum(0).to(torch.int32).to(dev)
    cfg = m3.linear_attention_config(q, k, v, batch_size=len(lengths), sequence_length=max(lengths),
                                     scale=SCALE)
    out = torch.empty(v.shape, dtype=v.dtype, device=dev)
    states = torch.empty(len(lengths), HEADS, HEAD_DIM, STATE, device=dev)
    ws = torch.empty(m3.m3_linear_attention_forward_workspace(cfg), dtype=torch.uint8, device=dev)
    m3.m3_linear_attention_forward(cfg, q, k, v, log_decay, offsets, None, out, states, ws)
    return out, states


def decode(x, w_in, weights, tabs, log_decay, positions, slots, pool):
    """One token of every sequence: rows [batch, WIDTH] -> outputs; the pool's slots move on."""
    q, k, v = split(x @ w_in)
    norm_rope_(q, k, weights, tabs, positions)
    cfg = m3.linear_attention_config(q, k, v, batch_size=len(x), sequence_length=1, scale=SCALE,
                                     num_slots=len(pool))
    out = torch.empty(v.shape, dtype=v.dtype, device=x.device)
    m3.m3_linear_attention_step(cfg, q, k, v, log_decay, slots, pool, out)
    return out


def serve():
    torch.manual_seed(0)
    lengths, more = [37, 200, 5, 1], 6
    tabs = tables(512)
    weights = [1 + 0.1 * torch.randn(STATE, device="cuda") for _ in range(2)]
    log_decay = -(2.0 ** -torch.linspace(1, 8, HEADS, device="cuda"))
    w_in = (torch.randn(WIDTH, 2 * QK + V, device="cuda") / 16).bfloat16()
    seqs = [torch.randn(n + more, WIDTH, device="cuda").bfloat16() for n in lengths]
    args = w_in, weights, tabs, log_decay

    whole, whole_states = prompts(torch.cat(seqs), *args, [n + more for n in lengths])
    _, states = prompts(torch.cat([s[:n] for s, n in zip(seqs, lengths)]), *args, lengths)
    pool = torch.zeros(8, HEADS, HEAD_DIM, STATE, device="cuda")
    slots = torch.tensor([6, 1, 3, 0], dtype=torch.int32, device="cuda")
    pool[slots.long()] = states
    worst = 0.0
    begin = torch.tensor([0] + [n + more for n in lengths]).cumsum(0)
    for t in range(more):
        x = torch.stack([s[n + t] for s, n in zip(seqs, lengths)])
        positions = torch.tensor(lengths, dtype=torch.int32, device="cuda") + t
        got = decode(x, *args, positions, slots, pool).double()
        want = torch.stack([whole[begin[i] + n + t] for i, n in enumerate(lengths)]).double()
        worst = max(worst, float((got - want).norm() / want.norm()))
    drift = float((pool[slots.long()] - whole_states).norm() / whole_states.norm())
    print(f"decoded {more} tokens of {len(lengths)} sequences: outputs within {worst:.1e} of the "
          f"prompt call's, states within {drift:.1e}")
    return worst


def train(steps=8):
    torch.manual_seed(1)
    batch, length = 2, 96
    tabs = tables(length)
    positions = torch.arange(length, dtype=torch.int32, device="cuda").repeat(batch)
    log_decay = -(2.0 ** -torch.linspace(1, 8, HEADS, device="cuda"))
    x = torch.randn(batch * length, WIDTH, device="cuda")
    target = torch.randn(batch * length, V, device="cuda")
    w_in = (torch.randn(WIDTH, 2 * QK + V, device="cuda") / 16).requires_grad_()
    weights = [torch.ones(STATE, device="cuda", requires_grad=True) for _ in range(2)]
    losses = []
    for _ in range(steps):
        q, k, v = split(x @ w_in)
        q, k = autograd.qk_norm_rope(q, k, *weights, *tabs, positions, ANGLES)
        out = autograd.linear_attention(q, k, v, log_decay, batch, length, scale=SCALE)
        loss = (out.reshape(batch * length, V) - target).square().mean()
        grads = torch.autograd.grad(loss, [w_in, *weights])
        with torch.no_grad():
            for p, g in zip([w_in, *weights], grads):
                p -= 0.2 * p.norm() / (g.norm() + 1e-9) * g * 0.1
        losses.append(float(loss.detach()))
    print(f"training: loss {losses[0]:.3f} -> {losses[-1]:.3f} in {steps} steps")
    return losses


def main():
    return serve(), train()


if __name__ == "__main__":
    main()

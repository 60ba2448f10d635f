"""The linear-attention operators of this package and what their calls cost.

Four entry points: the norm and position rotation of queries and keys
(forward and backward), and linear attention with a decay per head (prompts,
single tokens, backward). `run` calls them through the package where `own` is
true and computes them with elementary torch operations in 32 bits otherwise.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# cases

def _rope(name, rows, hq, hk, d, angles, dtype, backward, packed):
    return dict(name=name, op="rope", rows=rows, hq=hq, hk=hk, d=d, angles=angles, dtype=dtype,
                backward=backward, packed=packed)


def _prompt(name, batch, length, heads, groups, p, n, dtype, ragged, state, backward):
    return dict(name=name, op="prompt", batch=batch, length=length, heads=heads, groups=groups,
                p=p, n=n, dtype=dtype, ragged=ragged, state=state, backward=backward)


def _step(name, batch, slots, heads, groups, p, n, dtype):
    return dict(name=name, op="step", batch=batch, slots=slots, heads=heads, groups=groups, p=p,
                n=n, dtype=dtype)


def listed():
    return [
        # eight sequences decoding one token each: launch latency
        _rope("rope_decode_8", 8, 32, 32, 128, 32, "bf16", False, True),
        # the layer's prompt batch (8 x 2048 rows), queries and keys as views of packed rows
        _rope("rope_prompt_16k", 16384, 32, 32, 128, 64, "bf16", False, True),
        # training at the long-context layer: four key groups, half of the width rotated
        _rope("rope_backward_8k", 8192, 32, 4, 128, 32, "fp32", True, False),
        # one interactive sequence decoding one token
        _step("step_1", 1, 1, 32, 0, 64, 128, "bf16"),
        # the decode workload's batch with shared keys, states in a pool of slots
        _step("step_256", 256, 288, 32, 1, 64, 128, "fp32"),
        # the layer shape: eight prompts of 2048 tokens
        _prompt("prompt_layer", 8, 2048, 32, 0, 64, 128, "bf16", False, False, False),
        # the long-context shape, float32 with four groups of shared queries and keys
        _prompt("prompt_long_fp32", 2, 16384, 32, 4, 64, 128, "fp32", False, False, False),
        # one long document, square state
        _prompt("prompt_document", 1, 32768, 16, 0, 128, 128, "bf16", False, True, False),
        # a serving batch of short prompts of every length, continued from states
        _prompt("prompt_ragged", 24, 901, 20, 0, 80, 96, "bf16", True, True, False),
        # a training step of the layer shape
        _prompt("backward_layer", 8, 2048, 32, 0, 64, 128, "bf16", False, False, True),
        # training on long sequences with a square state, truncated back-propagation through states
        _prompt("backward_long", 2, 8192, 16, 0, 128, 128, "bf16", False, True, True),
        # a small float32 model with shared queries and keys
        _prompt("backward_fp32", 4, 1000, 8, 2, 64, 64, "fp32", False, True, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:  # again where a case would cost more than the largest listed one
        case = _drawn(rng)
        cost = work(case)
        if cost["bytes"] <= 730_000_000 and cost["flops"] <= 42_000_000_000:
            return case


def _drawn(rng):
    op = rng.choice(("rope", "prompt", "prompt", "step", "backward"))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    if op == "rope":
        d = rng.choice((32, 64, 80, 96, 128, 128, 192, 256, rng.randint(8, 256)))
        rows, hq = _log(rng, 1, 20000), rng.randint(1, 40)
        hk = rng.choice((hq, max(1, hq // 4), 1))
        rows = max(1, min(rows, 130_000_000 // (d * (hq + hk))))
        angles = rng.choice((0, d // 4, d // 2, d // 2, rng.randint(1, d // 2)))
        case = _rope("", rows, hq, hk, d, angles, dtype, rng.random() < 0.4, rng.random() < 0.5)
    else:
        p = rng.choice((16, 32, 64, 64, 80, 96, 128, 128, rng.randint(4, 128)))
        n = rng.choice((16, 32, 64, 96, 128, 128, 128, rng.randint(4, 128)))
        heads = rng.choice((1, 4, 8, 12, 16, 24, 32, 40))
        groups = rng.choice((0, 0, 1, max(1, heads // 4)))
        if op == "step":
            batch = max(1, min(_log(rng, 1, 400), 65_000_000 // (heads * p * n)))
            case = _step("", batch, batch + rng.randint(0, 9), heads, groups, p, n, dtype)
        else:
            back = op == "backward"
            most = min((1 if back else 3) * 1_000_000_000 // (heads * p * n),
                       (20_000_000 if back else 40_000_000) // (heads * (p + n)))
            length = max(1, min(_log(rng, 1, 30000), most))
            batch = max(1, min(_log(rng, 1, 24), most // length))
            case = _prompt("", batch, length, heads, groups, p, n, dtype, rng.random() < 0.4,
                           rng.random() < 0.5, back)
    del case["name"]
    return case


# ---------------------------------------------------------------------------
# inputs

def _lengths(case):
    """Lengths of a ragged batch: spread over 0 .. length, an empty one and the longest among them."""
    b, longest = case["batch"], case["length"]
    if not case["ragged"]:
        return [longest] * b
    return [longest if i == b - 1 else 0 if i == 1 else (longest * ((i * 7919) % 97)) // 97 + 1
            for i in range(b)]


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = dict(case=case)
    if case["op"] == "rope":
        rows, hq, hk, d, a = (case[x] for x in ("rows", "hq", "hk", "d", "angles"))
        if case["packed"]:  # q | k | v columns of one projection
            proj = _randn(gen, rows, (hq + hk + hk) * d).to(dt)
            s["q"] = proj[:, :hq * d].view(rows, hq, d)
            s["k"] = proj[:, hq * d:(hq + hk) * d].view(rows, hk, d)
        else:
            s["q"], s["k"] = _randn(gen, rows, hq, d).to(dt), _randn(gen, rows, hk, d).to(dt)
        s["wq"], s["wk"] = 1 + 0.1 * _randn(gen, d), 1 + 0.1 * _randn(gen, d)
        s["cos"] = s["sin"] = s["positions"] = None
        if a:
            freq = 10000.0 ** (-torch.arange(a, device="cuda", dtype=torch.float64) / a)
            ang = torch.arange(32768, device="cuda", dtype=torch.float64)[:, None] * freq
            s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
            s["positions"] = torch.randint(0, 32768, (rows,), generator=gen, device="cuda",
                                           dtype=torch.int32)
        s["outs"] = [torch.empty(rows, hq, d, device="cuda", dtype=dt),
                     torch.empty(rows, hk, d, device="cuda", dtype=dt)]
        if case["backward"]:
            s["dq"], s["dk"] = _randn(gen, rows, hq, d).to(dt), _randn(gen, rows, hk, d).to(dt)
            s["outs"] += [torch.empty(d, device="cuda"), torch.empty(d, device="cuda")]
    else:
        h, p, n = case["heads"], case["p"], case["n"]
        g = case["groups"] or h
        # unit-RMS queries and keys, as the norm before them leaves; log-spaced decays
        unit = lambda x: (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(dt)  # noqa: E731
        expo = torch.arange(h, device="cuda", dtype=torch.float32) / max(1, h - 1)
        s["log_decay"] = -(2.0 ** (-1.0 - 8.0 * expo))
        s["scale"] = 1.0 / math.sqrt(n)
        if case["op"] == "step":
            b, slots = case["batch"], case["slots"]
            s["q"], s["k"] = unit(_randn(gen, b, g, n)), unit(_randn(gen, b, g, n))
            s["v"] = _randn(gen, b, h, p).to(dt)
            s["state"] = _randn(gen, slots, h, p, n)
            order = torch.randperm(slots, generator=gen, device="cuda")[:b].to(torch.int32)
            if b > 2:
                order[b // 2] = -1  # a padding row of the batch
            s["slots"] = order
            s["out"] = torch.empty(b, h, p, device="cuda", dtype=dt)
        else:
            b, lens = case["batch"], _lengths(case)
            rows = sum(lens)
            s["q"], s["k"] = unit(_randn(gen, rows, g, n)), unit(_randn(gen, rows, g, n))
            s["v"] = _randn(gen, rows, h, p).to(dt)
            s["offsets"] = None
            if case["ragged"]:
                ends = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0)
                s["offsets"] = ends.to(torch.int32).cuda()
            s["initial"] = _randn(gen, b, h, p, n) if case["state"] else None
            if case["backward"]:
                s["dout"] = _randn(gen, rows, h, p).to(dt)
                s["dfinal"] = _randn(gen, b, h, p, n) if case["state"] else None
                s["grads"] = [torch.empty_like(s["q"]), torch.empty_like(s["k"]),
                              torch.empty_like(s["v"])]
                s["dinitial"] = torch.empty(b, h, p, n, device="cuda") if case["state"] else None
            else:
                s["out"] = torch.empty(rows, h, p, device="cuda", dtype=dt)
                s["final"] = torch.empty(b, h, p, n, device="cuda") if case["state"] else None
    _plan(s)
    return s


def _plan(s):
    """The configuration and workspace that a program keeps between calls."""
    if not own:
        return
    import selective_state_space_mamba3_gb300 as m3
    case = s["case"]
    if case["op"] == "rope":
        s["cfg"] = m3.qk_norm_rope_config(s["q"], s["k"], num_rope_angles=case["angles"],
                                          max_positions=32768, epsilon=1e-6)
        need = m3.m3_qk_norm_rope_backward_workspace(s["cfg"]) if case["backward"] else 0
    else:
        step = case["op"] == "step"
        s["cfg"] = m3.linear_attention_config(
            s["q"], s["k"], s["v"], batch_size=case["batch"],
            sequence_length=1 if step else case["length"], num_heads=case["heads"],
            num_groups=case["groups"], scale=s["scale"], num_slots=case["slots"] if step else 0)
        need = 0
        if not step:
            need = (m3.m3_linear_attention_backward_workspace if case["backward"] else
                    m3.m3_linear_attention_forward_workspace)(s["cfg"])
    s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")


# ---------------------------------------------------------------------------
# one pass

def run(s):
    case = s["case"]
    if own:
        import selective_state_space_mamba3_gb300 as m3
        if case["op"] == "rope":
            tables = (s["wq"], s["wk"], s["cos"], s["sin"], s["positions"])
            if case["backward"]:
                m3.m3_qk_norm_rope_backward(s["cfg"], s["q"], s["k"], *tables, s["dq"], s["dk"],
                                            *s["outs"], s["ws"])
            else:
                m3.m3_qk_norm_rope(s["cfg"], s["q"], s["k"], *tables, *s["outs"])
            return s["outs"]
        if case["op"] == "step":
            m3.m3_linear_attention_step(s["cfg"], s["q"], s["k"], s["v"], s["log_decay"],
                                        s["slots"], s["state"], s["out"])
            return [s["out"], s["state"]]
        if case["backward"]:
            m3.m3_linear_attention_backward(s["cfg"], s["dout"], s["q"], s["k"], s["v"],
                                            s["log_decay"], s["offsets"], s["initial"],
                                            s["dfinal"], *s["grads"], s["dinitial"], s["ws"])
            return [*s["grads"], s["dinitial"]]
        m3.m3_linear_attention_forward(s["cfg"], s["q"], s["k"], s["v"], s["log_decay"],
                                       s["offsets"], s["initial"], s["out"], s["final"], s["ws"])
        return [s["out"], s["final"]]
    if case["op"] == "rope":
        return _plain_rope_backward(s) if case["backward"] else _plain_rope(s)
    if case["op"] == "step":
        return _plain_step(s)
    return _plain_backward(s) if case["backward"] else _plain_prompt(s)


def _rotate(x, cos, sin, sign):
    a = cos.shape[-1]
    u, v, rest = x[..., :a], x[..., a:2 * a], x[..., 2 * a:]
    return torch.cat([u * cos - sign * v * sin, sign * u * sin + v * cos, rest], -1)


def _tables(s):
    if s["positions"] is None:
        return None, None
    at = s["positions"].long()
    return s["cos"][at][:, None], s["sin"][at][:, None]


def _plain_rope(s):
    cos, sin = _tables(s)
    outs = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        y = x.float()
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w
        outs.append((y if cos is None else _rotate(y, cos, sin, 1.0)).to(x.dtype))
    return outs


def _plain_rope_backward(s):
    cos, sin = _tables(s)
    dxs, dws = [], []
    for x, w, dy in ((s["q"], s["wq"], s["dq"]), (s["k"], s["wk"], s["dk"])):
        x32, g = x.float(), dy.float()
        if cos is not None:
            g = _rotate(g, cos, sin, -1.0)
        inv = torch.rsqrt(x32.square().mean(-1, keepdim=True) + 1e-6)
        xh = x32 * inv
        dws.append((g * xh).sum((0, 1)))
        g = g * w
        dxs.append((inv * (g - xh * (g * xh).mean(-1, keepdim=True))).to(x.dtype))
    return dxs + dws


def _plain_step(s):
    c = s["case"]
    rep = c["heads"] // (c["groups"] or c["heads"])
    q, k = (x.float().repeat_interleave(rep, 1) for x in (s["q"], s["k"]))
    v = s["v"].float()
    live = s["slots"] >= 0
    at = s["slots"].clamp(min=0).long()
    lam = s["log_decay"].exp()[:, None, None]
    new = s["state"][at] * lam + v[..., None] * k[..., None, :]
    out = (new * q[..., None, :]).sum(-1) * s["scale"]
    s["state"][at[live]] = new[live]
    return [torch.where(live[:, None, None], out, 0.0).to(s["v"].dtype), s["state"]]


def _padded(s, x):
    """[rows, heads, width] as float32 [batch, heads, length, width], zeros past a sequence's end."""
    c = s["case"]
    rep = c["heads"] // x.shape[1]
    if s["offsets"] is None:
        y = x.view(c["batch"], c["length"], *x.shape[1:]).float()
    else:
        off = s["offsets"].long()
        at = off[:-1, None] + torch.arange(c["length"], device="cuda")
        inside = at < off[1:, None]
        y = x[at.clamp(max=x.shape[0] - 1)].float() * inside[..., None, None]
    return y.repeat_interleave(rep, 2).transpose(1, 2)


def _rows(s, y, like):
    """The inverse of _padded; heads that share a group are summed."""
    c = s["case"]
    y = y.transpose(1, 2)
    rep = c["heads"] // like.shape[1]
    if rep > 1:
        y = y.reshape(*y.shape[:2], like.shape[1], rep, y.shape[-1]).sum(3)
    if s["offsets"] is None:
        return y.reshape(like.shape).to(like.dtype)
    off = s["offsets"].long()
    row = torch.arange(like.shape[0], device="cuda")
    b = torch.searchsorted(off, row, right=True) - 1
    return y[b, row - off[b]].to(like.dtype)


def _ends(s):
    c = s["case"]
    if s["offsets"] is None:
        return torch.full((c["batch"],), c["length"], device="cuda")
    return (s["offsets"][1:] - s["offsets"][:-1]).long()


def _causal(q, k, v, ld, state=None, chunk=64):
    """sum_{u<=t} lam^(t-u) (q_t.k_u) v_u + lam^(t+1) state q_t for float32 [B, H, L, width]:
    products inside chunks, and the chunks' states joined by one product with their decays."""
    b, h, n_tok, _ = q.shape
    pad = -n_tok % chunk
    q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, pad)).view(b, h, -1, chunk, x.shape[-1])
               for x in (q, k, v))
    i = torch.arange(chunk, device="cuda")
    gap = (i[:, None] - i).clamp(min=0)
    mask = torch.where(i[:, None] >= i, torch.exp(ld[:, None, None] * gap), 0.0)
    out = ((q @ k.transpose(-1, -2)) * mask[:, None]) @ v
    tail = torch.exp(ld[:, None] * (chunk - 1 - i))[:, None, :, None]
    sums = (v * tail).transpose(-1, -2) @ k  # [B, H, chunks, P, N]
    if state is None:
        state = torch.zeros_like(sums[:, :, 0])
    nc = sums.shape[2]
    c = torch.arange(nc, device="cuda")
    gap = chunk * (c[:, None] - 1 - c)
    w = torch.where(c[:, None] > c, torch.exp(ld[:, None, None] * gap.clamp(min=0)), 0.0)
    first = torch.exp(ld[:, None] * (chunk * c))[:, :, None]
    entry = torch.cat([first, w], 2) @ torch.cat([state[:, :, None], sums], 2).flatten(3)
    entry = entry.view(sums.shape)
    head = torch.exp(ld[:, None] * (i + 1))[:, None, :, None]
    out = out + head * (q @ entry.transpose(-1, -2))
    return out.flatten(2, 3)[:, :, :n_tok]


def _weights(s, power, inside):
    """lam^power where inside, else 0: [batch, heads, length, 1]."""
    e = torch.exp(s["log_decay"][:, None] * power[:, None].float())
    return torch.where(inside[:, None], e, 0.0)[..., None]


def _plain_prompt(s):
    ld, scale = s["log_decay"], s["scale"]
    q, k, v = (_padded(s, s[x]) for x in ("q", "k", "v"))
    out = _rows(s, scale * _causal(q, k, v, ld, s["initial"]), s["v"])
    if s["initial"] is None:
        return [out, None]
    ends = _ends(s)[:, None]
    left = ends - 1 - torch.arange(q.shape[2], device="cuda")
    final = (v * _weights(s, left.clamp(min=0), left >= 0)).transpose(-1, -2) @ k
    return [out, final + s["initial"] * torch.exp(ld * ends)[..., None, None]]


def _plain_backward(s):
    ld, scale = s["log_decay"], s["scale"]
    q, k, v, do = (_padded(s, s[x]) for x in ("q", "k", "v", "dout"))
    s0, ds = s["initial"], s["dfinal"]
    dq = scale * _causal(do, v, k, ld, None if s0 is None else s0.transpose(-1, -2))
    back = [x.flip(2) for x in (q, k, v, do)]
    dk = scale * _causal(back[2], back[3], back[0], ld).flip(2)
    dv = scale * _causal(back[1], back[0], back[3], ld).flip(2)
    ds0 = None
    if s0 is not None:
        t = torch.arange(q.shape[2], device="cuda")
        ends = _ends(s)[:, None]
        left = ends - 1 - t
        w = _weights(s, left.clamp(min=0), left >= 0)
        dk = dk + w * (v @ ds)
        dv = dv + w * (k @ ds.transpose(-1, -2))
        head = torch.exp(ld[:, None] * (t + 1))[..., None]
        ds0 = scale * (do * head).transpose(-1, -2) @ q
        ds0 = ds0 + ds * torch.exp(ld * ends)[..., None, None]
    return [_rows(s, dq, s["q"]), _rows(s, dk, s["k"]), _rows(s, dv, s["v"]), ds0]


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "rope":
        values = case["rows"] * case["d"] * (case["hq"] + case["hk"])
        table = case["rows"] * (8 * case["angles"] + 4)
        if case["backward"]:
            return {"bytes": 3 * e * values + table, "flops": 20 * values}
        return {"bytes": 2 * e * values + table, "flops": 8 * values}
    h, p, n = case["heads"], case["p"], case["n"]
    g = case["groups"] or h
    if case["op"] == "step":
        b = case["batch"]
        return {"bytes": b * (8 * h * p * n + e * (2 * g * n + 2 * h * p)),
                "flops": 5 * b * h * p * n}
    rows = sum(_lengths(case))
    states = 4 * case["batch"] * h * p * n if case["state"] else 0
    if case["backward"]:
        return {"bytes": e * rows * (4 * g * n + 3 * h * p) + 3 * states,
                "flops": 10 * rows * h * p * n}
    return {"bytes": e * rows * (2 * g * n + 2 * h * p) + 2 * states,
            "flops": 4 * rows * h * p * n}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, token by token

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s)
    h = case["heads"]
    rep = h // (case["groups"] or h)
    q, k = (s[x].double().repeat_interleave(rep, 1) for x in ("q", "k"))
    v = s["v"].double()
    lam = s["log_decay"].double().exp()[:, None, None]
    if case["op"] == "step":
        out, state = torch.zeros_like(v), s["state"].double()
        for i, at in enumerate(s["slots"].tolist()):
            if at >= 0:
                state[at] = lam * state[at] + v[i][:, :, None] * k[i][:, None, :]
                out[i] = s["scale"] * (state[at] @ q[i][:, :, None])[..., 0]
        return [out, state]
    lens = _lengths(case)
    begin = [sum(lens[:i]) for i in range(len(lens))]
    order = sorted(range(len(lens)), key=lambda i: -lens[i])  # the live ones stay a prefix
    first = torch.tensor([begin[i] for i in order], device="cuda")
    last = torch.tensor([begin[i] + lens[i] - 1 for i in order], device="cuda")
    live = [sum(1 for i in order if lens[i] > t) for t in range(max(lens))]
    back = torch.tensor(order, device="cuda")
    zero = torch.zeros(len(lens), h, case["p"], case["n"], device="cuda", dtype=torch.float64)
    state = zero.clone() if s["initial"] is None else s["initial"].double()[back]
    if not case["backward"]:
        out = torch.zeros_like(v)
        for t, m in enumerate(live):
            at = first[:m] + t
            state[:m] = lam * state[:m] + v[at][..., :, None] * k[at][..., None, :]
            out[at] = s["scale"] * (state[:m] @ q[at][..., None])[..., 0]
        return [out, None if s["initial"] is None else _unsort(state, back)]
    do = s["dout"].double()
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for t, m in enumerate(live):
        at = first[:m] + t
        state[:m] = lam * state[:m] + v[at][..., :, None] * k[at][..., None, :]
        dq[at] = s["scale"] * (do[at][..., None, :] @ state[:m])[..., 0, :]
    grad = zero if s["dfinal"] is None else s["dfinal"].double()[back]  # d loss / d state after a token
    for t, m in enumerate(live):
        at = last[:m] - t
        grad[:m] = grad[:m] + s["scale"] * do[at][..., :, None] * q[at][..., None, :]
        dk[at] = (v[at][..., None, :] @ grad[:m])[..., 0, :]
        dv[at] = (grad[:m] @ k[at][..., None])[..., 0]
        grad[:m] = lam * grad[:m]
    if rep > 1:
        dq, dk = (x.view(x.shape[0], h // rep, rep, -1).sum(2) for x in (dq, dk))
    return [dq, dk, dv, None if s["dfinal"] is None else _unsort(grad, back)]


def _unsort(state, back):
    out = torch.empty_like(state)
    out[back] = state
    return out


def _exact_rope(s):
    a, d = s["case"]["angles"], s["case"]["d"]
    turn = None
    if a:
        at = s["positions"].long()
        turn = torch.complex(s["cos"][at].double(), s["sin"][at].double())[:, None]
    outs, weights = [], []
    for x, w, dy in ((s["q"], s["wq"], s.get("dq")), (s["k"], s["wk"], s.get("dk"))):
        x, w = x.double(), w.double()
        norm = torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / d + 1e-6)
        y = (x / norm * w) if dy is None else dy.double().clone()
        if a:
            z = torch.complex(y[..., :a].contiguous(), y[..., a:2 * a].contiguous())
            z = z * (turn if dy is None else turn.conj())
            y[..., :a], y[..., a:2 * a] = z.real, z.imag
        if dy is not None:
            weights.append((y * x / norm).sum(0).sum(0))
            dot = torch.einsum("rhd,rhd->rh", y * w, x)[..., None]
            y = y * w / norm - x * dot / (d * norm ** 3)
        outs.append(y)
    return outs + weights

"""Cases for timing and checking the transformer-block operators: attention over packed
sequences, residual addition with root-mean-square norm, and rotary positions with several axes.

A case is a dict of plain values.  ``prepare`` makes its tensors on the GPU from a seed,
``run`` makes one pass: with the library's calls where ``own`` is true, else in a plain form of
elementary torch operations in 32 bits.  ``exact`` gives the same outputs in 64 bits, ``work``
the bytes and operations that a pass cannot do without.

Features follow the layer's layout [N, C, G] with the group axis fastest.  A head is ``D``
consecutive features (D / G channels with all their group elements).
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
E4M3_MAX = 448.0
EPS = 1e-6
BASE = 100.0


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # latency: the smallest layer of the workloads (16 channels, p4), one sequence, fp32
        {"name": "attn_tiny_train_f32", "op": "attn", "mode": "train", "type": "f32", "G": 4, "D": 64, "heads": 1,
         "kv_heads": 1, "batch": 1, "q_len": 256, "k_len": 256, "ragged": 0, "causal": False},
        # windows of 7 x 7 tokens over 64 maps of 56 x 56 (p4, 96 channels, 3 heads of 32 channels)
        {"name": "attn_windows_fwd_bf16", "op": "attn", "mode": "fwd", "type": "bf16", "G": 4, "D": 128, "heads": 3,
         "kv_heads": 3, "batch": 4096, "q_len": 49, "k_len": 49, "ragged": 0, "causal": False},
        # inference over 32 whole maps of 28 x 28 tokens (p8, 64 channels, 8 heads of 8 channels)
        {"name": "attn_maps_fwd_bf16", "op": "attn", "mode": "fwd", "type": "bf16", "G": 8, "D": 64, "heads": 8,
         "kv_heads": 8, "batch": 32, "q_len": 784, "k_len": 784, "ragged": 0, "causal": False},
        # the training step of the same
        {"name": "attn_maps_train_bf16", "op": "attn", "mode": "train", "type": "bf16", "G": 8, "D": 64, "heads": 8,
         "kv_heads": 8, "batch": 32, "q_len": 784, "k_len": 784, "ragged": 0, "causal": False},
        # packed sequences of different lengths, causal, shared key and value heads, fp16
        {"name": "attn_ragged_fwd_f16", "op": "attn", "mode": "fwd", "type": "f16", "G": 4, "D": 128, "heads": 6,
         "kv_heads": 2, "batch": 12, "q_len": 4096, "k_len": 4096, "ragged": 5, "causal": True},
        # the largest: training on one long causal scan of a map (p4, 192 channels, 6 heads of 32 channels)
        {"name": "attn_long_train_bf16", "op": "attn", "mode": "train", "type": "bf16", "G": 4, "D": 128, "heads": 6,
         "kv_heads": 6, "batch": 1, "q_len": 16384, "k_len": 16384, "ragged": 0, "causal": True},
        # one pooling query for each of 8 maps of 128 x 128 tokens
        {"name": "attn_one_query_bf16", "op": "attn", "mode": "fwd", "type": "bf16", "G": 8, "D": 64, "heads": 8,
         "kv_heads": 2, "batch": 8, "q_len": 1, "k_len": 16384, "ragged": 0, "causal": False},
        # norm of the widest token batch of the workloads, forward and gradients
        {"name": "norm_train_bf16", "op": "norm", "mode": "train", "type": "bf16", "G": 4, "C": 96, "N": 200704},
        # norm with 8-bit outputs (p8)
        {"name": "norm_fp8_bf16", "op": "norm", "mode": "fp8", "type": "bf16", "G": 8, "C": 64, "N": 25088},
        # latency: the norm of one map of 14 x 14 tokens
        {"name": "norm_small_fwd_f16", "op": "norm", "mode": "fwd", "type": "f16", "G": 4, "C": 96, "N": 196},
        # rotation of queries and keys inside a joint projection, by row and column (p4)
        {"name": "rope_maps_bf16", "op": "rope", "type": "bf16", "G": 4, "D": 128, "heads": 6, "rows": 9, "axes": 2,
         "N": 200704, "inverse": False, "far": 56},
        # the gradient of a rotation by time, row and column of a short clip (C16), 8 frames of 14 x 14
        {"name": "rope_clip_grad_f16", "op": "rope", "type": "f16", "G": 16, "D": 128, "heads": 8, "rows": 8, "axes": 3,
         "N": 1568, "inverse": True, "far": 14},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "norm", "rope"])
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    G = rng.choice([2, 4, 8, 16])
    if op == "norm":
        step = max(1, 8 // G)
        C = step * max(1, _log(rng, 8, 4096) // (G * step))
        return {"op": "norm", "mode": rng.choice(["fwd", "fp8", "train"]), "type": kind, "G": G, "C": C,
                "N": min(_log(rng, 1, 200704), 200704 * 384 // (C * G))}
    if op == "rope":
        D = 2 * G * max(1, _log(rng, 16, 128) // (2 * G))
        axes = rng.randint(1, min(3, D // G // 2))
        heads = rng.randint(1, 12)
        rows = heads + rng.choice([0, 1, 4])
        return {"op": "rope", "type": kind, "G": G, "D": D, "heads": heads, "rows": rows, "axes": axes,
                "N": min(_log(rng, 1, 200704), 200704 * 768 // (rows * D)), "inverse": rng.random() < 0.5,
                "far": _log(rng, 1, 100000)}
    D = 8 * rng.randint(2, 16)
    G = rng.choice([g for g in (2, 4, 8, 16) if D % g == 0])
    kv_heads = rng.randint(1, 4)
    heads = kv_heads * rng.choice([1, 1, 2, 3])
    shape = rng.choice(["windows", "maps", "ragged", "cross", "long", "query"])
    causal = rng.random() < 0.5
    if shape == "windows":
        batch, q_len = _log(rng, 16, 4096), rng.randint(1, 64)
        k_len, ragged, causal = q_len, 0, False
    elif shape == "maps":
        batch, q_len = _log(rng, 1, 32), _log(rng, 65, 1024)
        k_len, ragged = q_len, 0
    elif shape == "ragged":
        batch, q_len = rng.randint(2, 16), _log(rng, 64, 4096)
        k_len, ragged = q_len, rng.randint(1, 1 << 20)
    elif shape == "cross":
        batch, q_len, k_len = rng.randint(1, 16), _log(rng, 16, 2048), _log(rng, 16, 2048)
        ragged = rng.randint(1, 1 << 20)
    elif shape == "long":
        batch, q_len = 1, _log(rng, 4096, 16384)
        k_len, ragged = q_len, 0
    else:
        batch, q_len, k_len, ragged, causal = rng.randint(1, 16), 1, _log(rng, 256, 32768), 0, False
    mode = "fwd" if shape == "query" else rng.choice(["fwd", "train"])
    most = (1 << 28) if kind == "f32" else 6 * 16384 * 16384
    while batch * heads * q_len * k_len > most or batch * heads * max(q_len, k_len) * D > 200704 * 384:
        if batch > 1:
            batch -= -(-batch // 4)
        elif heads > kv_heads:
            heads = kv_heads
        elif kv_heads > 1:
            heads = kv_heads = kv_heads - 1
        else:
            q_len, k_len = (q_len * 3 + 3) // 4, (k_len * 3 + 3) // 4
    return {"op": "attn", "mode": mode, "type": kind, "G": G, "D": D, "heads": heads, "kv_heads": kv_heads,
            "batch": batch, "q_len": q_len, "k_len": k_len, "ragged": ragged, "causal": causal}


def lengths(case):
    """(query lengths, key lengths) of the packed sequences; `ragged` is 0 or what they are made from."""
    B, Lq, Lk = case["batch"], case["q_len"], case["k_len"]
    if not case["ragged"]:
        return [Lq] * B, [Lk] * B
    rng = random.Random(case["ragged"])
    if Lq == Lk:                       # self-attention: from a single token to the longest
        q = [_log(rng, 1, Lq) for _ in range(B)]
        q[rng.randrange(B)] = Lq
        return q, list(q)
    return [rng.randint(0, Lq) for _ in range(B)], [rng.randint(0, Lk) for _ in range(B)]


def sections(pairs, axes):
    """How many channel pairs of a head turn with each axis: as even as possible, the first ones more."""
    return [pairs // axes + (1 if a < pairs % axes else 0) for a in range(axes)]


# ---------------------------------------------------------------------------------- the inputs
def _offsets(lens, device):
    t = torch.zeros(len(lens) + 1, dtype=torch.int64)
    t[1:] = torch.tensor(lens, dtype=torch.int64).cumsum(0)
    return t.to(torch.int32).to(device)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    T = TYPES[case["type"]]

    def normal(*shape, std=1.0, dtype=T):
        return (torch.randn(*shape, device=dev, generator=g) * std).to(dtype)

    s = {"case": case}
    G = case["G"]
    if case["op"] == "norm":
        N, C = case["N"], case["C"]
        s["x"], s["residual"] = normal(N, C, G), normal(N, C, G, std=2.0)
        s["weight"] = (1 + 0.2 * torch.randn(C, device=dev, generator=g)).to(T)
        if case["mode"] == "train":
            s["dy"], s["dsum"] = normal(N, C, G), normal(N, C, G)
        return s
    if case["op"] == "rope":
        N, D = case["N"], case["D"]
        s["joint"] = normal(N, case["rows"] * D // G, G)
        s["x"] = s["joint"][:, :case["heads"] * D // G]
        s["positions"] = torch.randint(0, case["far"], (N, case["axes"]), device=dev, generator=g, dtype=torch.int32)
        s["sections"] = sections(D // G // 2, case["axes"])
        return s
    q_lens, k_lens = lengths(case)
    Nq, Nk, Dh = sum(q_lens), sum(k_lens), case["D"] // G
    H, Hk = case["heads"], case["kv_heads"]
    if q_lens == k_lens:               # self-attention reads its tensors out of one joint projection
        joint = normal(Nq, (H + 2 * Hk) * Dh, G)
        s["q"], s["k"], s["v"] = joint[:, :H * Dh], joint[:, H * Dh:(H + Hk) * Dh], joint[:, (H + Hk) * Dh:]
    else:
        s["q"], s["k"], s["v"] = normal(Nq, H * Dh, G), normal(Nk, Hk * Dh, G), normal(Nk, Hk * Dh, G)
    if case["mode"] == "train":
        s["do"] = normal(Nq, H * Dh, G)
    s["q_offsets"], s["k_offsets"] = _offsets(q_lens, dev), _offsets(k_lens, dev)
    s["q_most"], s["k_most"] = max(q_lens), max(k_lens)
    return s


# ---------------------------------------------------------------------------------- the passes
def run(s):
    case = s["case"]
    if case["op"] == "norm":
        return _own_norm(s) if own else _plain_norm(s)
    if case["op"] == "rope":
        return _own_rope(s) if own else _plain_rope(s)
    return _own_attn(s) if own else _plain_attn(s)


def _own_norm(s):
    import cyclic_group_dft_b200 as eq
    mode = s["case"]["mode"]
    if mode == "fp8":
        y, scale, total = eq.eqlin_add_rmsnorm_fp8(s["x"], s["residual"], s["weight"], eps=EPS)
        return {"y": y, "scale": scale, "sum": total}
    y, total = eq.eqlin_add_rmsnorm(s["x"], s["residual"], s["weight"], eps=EPS)
    out = {"y": y, "sum": total}
    if mode == "train":
        out["dx"], out["dweight"] = eq.eqlin_rmsnorm_backward(s["dy"], total, s["weight"], dsum=s["dsum"], eps=EPS)
    return out


def _own_rope(s):
    import cyclic_group_dft_b200 as eq
    case = s["case"]
    return {"y": eq.eqlin_rope(s["x"], s["positions"], heads=case["heads"], sections=s["sections"], base=BASE,
                               inverse=case["inverse"])}


def _own_attn(s):
    import cyclic_group_dft_b200 as eq
    case = s["case"]
    how = {"heads": case["heads"], "kv_heads": case["kv_heads"], "q_offsets": s["q_offsets"],
           "k_offsets": s["k_offsets"], "causal": case["causal"]}
    o, lse = eq.eqlin_attention_forward(s["q"], s["k"], s["v"], **how)
    out = {"o": o, "lse": lse}
    if case["mode"] == "train":
        q, k, v = s["q"], s["k"], s["v"]
        grads = None
        if q.stride(0) != q.shape[1] * q.shape[2]:      # the gradient of the joint projection, in one tensor
            joint = torch.empty(q.shape[0], q.stride(0) // q.shape[2], q.shape[2], dtype=q.dtype, device=q.device)
            a, b = q.shape[1], q.shape[1] + k.shape[1]
            grads = (joint[:, :a], joint[:, a:b], joint[:, b:])
        out["dq"], out["dk"], out["dv"] = eq.eqlin_attention_backward(s["do"], q, k, v, o, lse, grads=grads, **how)
    return out


def _plain_norm(s):
    T = s["x"].dtype
    w = s["weight"].float()[None, :, None]
    r = s["x"].float() + s["residual"].float()
    y = r * torch.rsqrt((r * r).mean((1, 2), keepdim=True) + EPS) * w
    out = {"y": y.to(T), "sum": r.to(T)}
    if s["case"]["mode"] == "fp8":
        top = y.abs().amax((1, 2))
        out["scale"] = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
        out["y"] = (y / out["scale"][:, None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    if s["case"]["mode"] == "train":
        r = out["sum"].float()         # the backward pass has the stored sum
        rstd = torch.rsqrt((r * r).mean((1, 2), keepdim=True) + EPS)
        dy, unit = s["dy"].float(), r * rstd
        wdy = dy * w
        dx = rstd * (wdy - unit * (wdy * unit).mean((1, 2), keepdim=True)) + s["dsum"].float()
        out["dx"] = dx.to(T)
        out["dweight"] = (dy * unit).double().sum((0, 2)).float()
    return out


def _plain_rope(s):
    case, x = s["case"], s["x"]
    N, D, G, H = case["N"], case["D"], case["G"], case["heads"]
    cos, sin = _turns(s, torch.float32)
    v = x.float().reshape(N, H, 2, D // G // 2, G)
    a, b = v[:, :, 0], v[:, :, 1]
    if case["inverse"]:
        sin = -sin
    y = torch.stack([a * cos - b * sin, b * cos + a * sin], 2)
    return {"y": y.reshape(x.shape).to(x.dtype)}


def _turns(s, dtype):
    """cos and sin [N, 1, pairs, 1] of position times frequency, the angle in 64 bits."""
    angles = torch.cat([s["positions"][:, a:a + 1].double()
                        * (BASE ** (-torch.arange(n, device=s["positions"].device).double() / n))
                        for a, n in enumerate(s["sections"])], 1)[:, None, :, None]
    return angles.cos().to(dtype), angles.sin().to(dtype)


def _rows(offsets, most):
    """Row of token i of sequence b in the packed tensors, and whether there is one: [batch, most]."""
    i = torch.arange(most, device=offsets.device)
    start, end = offsets[:-1].long(), offsets[1:].long()
    rows = start[:, None] + i[None, :]
    there = rows < end[:, None]
    return torch.where(there, rows, torch.zeros_like(rows)), there


def _plain_attn(s):
    case = s["case"]
    H, Hk, D, T = case["heads"], case["kv_heads"], case["D"], s["q"].dtype
    scale = 1 / math.sqrt(D)
    qr, q_there = _rows(s["q_offsets"], s["q_most"])
    kr, k_there = _rows(s["k_offsets"], s["k_most"])
    B, Lq, Lk = len(qr), s["q_most"], s["k_most"]

    def taken(t, rows, there, heads):      # [batch, kv_heads, heads of the group * length, D]
        if len(t) == 0:
            return torch.zeros(B, Hk, heads // Hk * rows.shape[1], D, device=t.device)
        t = t.reshape(len(t), heads, D)[rows].float() * there[:, :, None, None]
        return t.permute(0, 2, 1, 3).reshape(B, Hk, -1, D)

    def put(t, rows, there, heads, n):     # back into packed rows
        t = t.reshape(B, heads, rows.shape[1], D).permute(0, 2, 1, 3)
        out = torch.zeros(n, heads, D, device=t.device)
        out[rows[there]] = t[there]
        return out.to(T)

    q, k, v = taken(s["q"], qr, q_there, H), taken(s["k"], kr, k_there, Hk), taken(s["v"], kr, k_there, Hk)
    seen = q_there[:, :, None] & k_there[:, None, :]
    if case["causal"]:                     # the last query of a sequence sees its last key
        behind = k_there.sum(1) - q_there.sum(1)
        i, j = torch.arange(Lq, device=q.device), torch.arange(Lk, device=q.device)
        seen &= j[None, None, :] <= i[None, :, None] + behind[:, None, None]
    shape = (B, Hk, H // Hk, Lq, Lk)
    w = (q @ k.transpose(2, 3) * scale).reshape(shape).masked_fill_(~seen[:, None, None], -math.inf)
    top = w.amax(-1, keepdim=True)
    w = w.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = w.sum(-1, keepdim=True)
    w = w.div_(torch.where(total > 0, total, torch.ones_like(total))).reshape(B, Hk, -1, Lk)
    lse = (top + total.log()).reshape(B, H, Lq).permute(0, 2, 1)
    o = w @ v
    flat = torch.empty(len(s["q"]), H, device=q.device)
    flat[qr[q_there]] = lse[q_there]
    out = {"o": put(o, qr, q_there, H, len(s["q"])).reshape(s["q"].shape), "lse": flat.t().contiguous()}
    if case["mode"] == "train":
        do = taken(s["do"], qr, q_there, H)
        dv = w.transpose(2, 3) @ do
        dw = do @ v.transpose(2, 3)
        dw = dw.sub_((do * o).sum(-1, keepdim=True)).mul_(w).mul_(scale)
        del w
        out["dq"] = put(dw @ k, qr, q_there, H, len(s["q"])).reshape(s["q"].shape)
        out["dk"] = put(dw.transpose(2, 3) @ q, kr, k_there, Hk, len(s["k"])).reshape(s["k"].shape)
        out["dv"] = put(dv, kr, k_there, Hk, len(s["k"])).reshape(s["v"].shape)
    return out


# ------------------------------------------------------------------------------ the definition
def work(case):
    e = BYTES[case["type"]]
    if case["op"] == "norm":
        n, N = case["N"] * case["C"] * case["G"], case["N"]
        moved, flops = (4 * n * e, 6 * n) if case["mode"] == "fwd" else (n * (3 * e + 1) + 4 * N, 8 * n)
        if case["mode"] == "train":        # x, residual, dy, dsum in; y, sum, dx out
            moved, flops = 7 * n * e + 4 * case["C"], 18 * n
        return {"bytes": moved + case["C"] * e, "flops": flops}
    if case["op"] == "rope":
        n = case["N"] * case["heads"] * case["D"]
        return {"bytes": 2 * n * e + 4 * case["N"] * case["axes"], "flops": 3 * n}
    q_lens, k_lens = lengths(case)
    H, Hk, D, Nq, Nk = case["heads"], case["kv_heads"], case["D"], sum(q_lens), sum(k_lens)
    pairs = 0
    for a, b in zip(q_lens, k_lens):
        if not case["causal"]:
            pairs += a * b
        else:                              # query i sees max(0, i + 1 + b - a) keys
            n = min(a, b)
            pairs += n * (b - n) + n * (n + 1) // 2
    moved = (2 * Nq * H + 2 * Nk * Hk) * D * e + 4 * H * Nq + 8 * (case["batch"] + 1)
    flops = 4 * pairs * H * D
    if case["mode"] == "train":
        moved += (2 * Nq * H + 2 * Nk * Hk) * D * e
        flops += 10 * pairs * H * D
    return {"bytes": moved, "flops": flops}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(case, s)
    if case["op"] == "rope":
        cos, sin = _exact_turns(case, s)
        half = case["D"] // 2
        x = s["x"].double().reshape(case["N"], case["heads"], case["D"])
        other = torch.cat([-x[..., half:], x[..., :half]], -1)
        return {"y": (x * cos + other * (-sin if case["inverse"] else sin)).reshape(s["x"].shape)}
    return _exact_attn(case, s)


def _exact_turns(case, s):
    """cos and sin [N, 1, D] of every feature of a head."""
    pairs, G, at = case["D"] // case["G"] // 2, case["G"], []
    for a, n in enumerate(s["sections"]):
        at += [(a, math.exp(-j / n * math.log(BASE))) for j in range(n)]
    axis = torch.tensor([a for a, _ in at], device=s["x"].device)
    freq = torch.tensor([f for _, f in at], dtype=torch.float64, device=s["x"].device)
    angle = s["positions"].double()[:, axis] * freq
    angle = angle.repeat_interleave(G, 1).repeat(1, 2)[:, None, :]
    assert angle.shape[-1] == 2 * pairs * G
    return torch.cos(angle), torch.sin(angle)


def _exact_norm(case, s):
    n, C, G = case["N"], case["C"], case["G"]
    r = (s["x"].double() + s["residual"].double()).reshape(n, C * G)
    w = s["weight"].double().repeat_interleave(G)
    norm = torch.sqrt(r.pow(2).sum(1, keepdim=True) / (C * G) + EPS)
    y = r / norm * w
    shape = (n, C, G)
    if case["mode"] == "fp8":
        top = y.abs().max(1, keepdim=True).values
        scale = torch.where(top == 0, torch.ones_like(top), top / E4M3_MAX)
        return {"y": (y / scale).reshape(shape), "scale": scale[:, 0], "sum": r.reshape(shape)}
    out = {"y": y.reshape(shape), "sum": r.reshape(shape)}
    if case["mode"] == "train":
        r = r.to(TYPES[case["type"]]).double()
        norm = torch.sqrt(r.pow(2).sum(1, keepdim=True) / (C * G) + EPS)
        dy, dsum = s["dy"].double().reshape(n, C * G), s["dsum"].double().reshape(n, C * G)
        inner = (dy * w * r).sum(1, keepdim=True) / (C * G)
        out["dx"] = (dsum + dy * w / norm - r * inner / norm.pow(3)).reshape(shape)
        out["dweight"] = (dy * r / norm).sum(0).reshape(C, G).sum(1)
    return out


def _exact_attn(case, s):
    q_lens, k_lens = lengths(case)
    H, Hk, D = case["heads"], case["kv_heads"], case["D"]
    group, train = H // Hk, case["mode"] == "train"
    if case["batch"] > 64:                 # many sequences are of one length: a few batched steps
        step = max(1, (1 << 26) // (H * case["q_len"] * case["k_len"]))
        parts = [(b, min(step, case["batch"] - b)) for b in range(0, case["batch"], step)]
    else:
        parts = [(b, 1) for b in range(case["batch"])]
    dev = s["q"].device
    out = {"o": torch.zeros(len(s["q"]), H, D, dtype=torch.float64, device=dev),
           "lse": torch.full((H, len(s["q"])), -math.inf, dtype=torch.float64, device=dev)}
    if train:
        out["dq"] = torch.zeros_like(out["o"])
        out["dk"] = torch.zeros(len(s["k"]), Hk, D, dtype=torch.float64, device=dev)
        out["dv"] = torch.zeros_like(out["dk"])

    def part(t, at, n, length, head):      # [n, length, D]
        return t[at:at + n * length].reshape(n * length, -1, D)[:, head].reshape(n, length, D).double()

    qs, ks = [0], [0]
    for a, b in zip(q_lens, k_lens):
        qs.append(qs[-1] + a)
        ks.append(ks[-1] + b)
    for b, n in parts:
        Lq, Lk, q0, k0 = q_lens[b], k_lens[b], qs[b], ks[b]
        if Lq == 0 or Lk == 0:
            continue
        for h in range(H):
            g = h // group
            q, k, v = part(s["q"], q0, n, Lq, h), part(s["k"], k0, n, Lk, g), part(s["v"], k0, n, Lk, g)
            score = torch.einsum("nid,njd->nij", q, k) / math.sqrt(D)
            if case["causal"]:
                hidden = torch.ones(Lq, Lk, dtype=torch.bool, device=dev).triu(Lk - Lq + 1)
                score.masked_fill_(hidden, -math.inf)
            lse = torch.logsumexp(score, -1)
            p = torch.exp(score - lse[..., None].masked_fill(lse[..., None] == -math.inf, 0.0))
            del score
            o = torch.einsum("nij,njd->nid", p, v)
            out["o"][q0:q0 + n * Lq, h] = o.reshape(-1, D)
            out["lse"][h, q0:q0 + n * Lq] = lse.reshape(-1)
            if train:
                do = part(s["do"], q0, n, Lq, h)
                out["dv"][k0:k0 + n * Lk, g] += torch.einsum("nij,nid->njd", p, do).reshape(-1, D)
                ds = torch.einsum("nid,njd->nij", do, v)
                ds -= (do * o).sum(-1)[..., None]
                ds *= p
                ds /= math.sqrt(D)
                out["dq"][q0:q0 + n * Lq, h] = torch.einsum("nij,njd->nid", ds, k).reshape(-1, D)
                out["dk"][k0:k0 + n * Lk, g] += torch.einsum("nij,nid->njd", ds, q).reshape(-1, D)
    for name, like in (("o", "q"), ("dq", "q"), ("dk", "k"), ("dv", "v")):
        if name in out:
            out[name] = out[name].reshape(s[like].shape)
    return out

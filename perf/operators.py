"""The operators around the MoE layer, as they are measured: the product with
4-bit weights, the norms before and after a block, and the log probabilities
of given tokens.

listed() and draw() give the cases, prepare() the inputs of one, run() one
pass: in plain torch operations, or (own) through the library's calls.
"""
from __future__ import annotations

import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------- cases

def _q4(name, m, n, k, group, zeros=False, x="bf16", s="f16", out="f32", pad=0):
    """out[m, n] from 4-bit weights [n, k]; pad: extra values of row pitch in x and out"""
    c = {"op": "q4", "m": m, "n": n, "k": k, "group": group, "zeros": zeros, "x": x, "s": s, "out": out, "pad": pad}
    return {"name": name, **c} if name else c


def _norm(name, m, dim, kind, y, h, x, gate, w="f32", post=True, gate_group=1):
    """gate: none, channel [dim], row [ceil(m / gate_group), dim] or token [m]"""
    c = {"op": "norm", "m": m, "dim": dim, "kind": kind, "y": y, "h": h, "x": x, "gate": gate, "w": w, "post": post,
         "gate_group": gate_group}
    return {"name": name, **c} if name else c


def _lp(name, m, vocab, t, top, mask=False, temp=1.0, pad=0):
    c = {"op": "logprob", "m": m, "vocab": vocab, "type": t, "top": top, "mask": mask, "temp": temp, "pad": pad}
    return {"name": name, **c} if name else c


def listed():
    return [
        # a narrow projection of one token (a low-rank query or a gate): latency counts
        _q4("q4_narrow_m1", 1, 512, 5120, 128),
        # one token through a dense down projection as wide as an expert's, asymmetric codes
        _q4("q4_down_m1", 1, 5120, 2304, 64, zeros=True, s="bf16", out="bf16"),
        # one token's logits over a 128 Ki vocabulary: the largest read of a decode step
        _q4("q4_head_m1", 1, 131072, 5120, 128),
        # a decode batch of eight through a fused gate and up projection, small groups
        _q4("q4_gateup_m8", 8, 4608, 5120, 32, x="f16", out="f16"),
        # five sequences, an odd vocabulary, a width that is no multiple of the group, padded rows
        _q4("q4_ragged_m5", 5, 50001, 2336, 128, zeros=True, pad=24),
        # the logits of a prompt chunk that is scored
        _q4("q4_head_m512", 512, 131072, 5120, 128),
        # one decode token: the MoE output (f32) onto the residual, then the next block's norm
        _norm("norm_m1", 1, 5120, "rms", "f32", "bf16", "bf16", "channel"),
        # a long prefill chunk with an f32 residual stream
        _norm("norm_m4096", 4096, 5120, "rms", "f32", "f32", "bf16", "token"),
        # layer norms at an odd width, a gate row per request of 37 tokens
        _norm("norm_odd_m333", 333, 2305, "layer", "bf16", "bf16", "f16", "row", w="bf16", gate_group=37),
        # one decode token: the answer with 20 alternatives, under a grammar's mask
        _lp("logprob_m1_masked", 1, 131072, "f32", 20, mask=True, temp=0.7),
        # the scored prompt chunk
        _lp("logprob_m512", 512, 131072, "f32", 20),
        # bf16 logits of an odd vocabulary (rows start at any 2-byte address), five alternatives, many ties
        _lp("logprob_bf16_m1000", 1000, 50001, "bf16", 5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["q4", "q4", "norm", "logprob"])
    if op == "q4":
        m = rng.randint(1, 8) if rng.random() < 0.7 else _log(rng, 9, 512)
        k = 32 * _log(rng, 8, 256)
        n = _log(rng, 64, min(131072, 131072 * 5120 // k))
        return _q4(None, m, n, k, rng.choice([32, 64, 128]), rng.random() < 0.5, rng.choice(["bf16", "f16"]),
                   rng.choice(["bf16", "f16"]), rng.choice(["f32", "bf16", "f16"]), rng.choice([0, 8, 24]))
    if op == "norm":
        dim = _log(rng, 256, 7680)
        dim = dim if rng.random() < 0.3 else max(256, dim // 64 * 64)
        m = _log(rng, 1, min(4096, 4096 * 5120 // dim))
        return _norm(None, m, dim, rng.choice(["rms", "layer"]), rng.choice(["f32", "bf16", "f16"]),
                     rng.choice(["f32", "bf16"]), rng.choice(["bf16", "f16"]),
                     rng.choice(["none", "channel", "row", "token"]), rng.choice(["f32", "bf16"]), rng.random() < 0.8,
                     rng.choice([1, 7, 64]))
    vocab = _log(rng, 1000, 131072)
    m = _log(rng, 1, min(1000, 512 * 131072 // vocab))
    return _lp(None, m, vocab, rng.choice(["f32", "bf16", "f16"]), rng.choice([0, 1, 5, 20]), rng.random() < 0.4,
               rng.choice([0.7, 1.0, 1.3]), rng.choice([0, 0, 3, 8]))


def work(c):
    if c["op"] == "q4":
        m, n, k = c["m"], c["n"], c["k"]
        groups = -(-k // c["group"])
        return {"bytes": n * k // 2 + n * groups * (3 if c["zeros"] else 2) + m * k * 2 + m * n * SIZE[c["out"]],
                "flops": 2 * m * n * k}
    if c["op"] == "norm":
        m, d = c["m"], c["dim"]
        gate = {"none": 0, "channel": d, "row": -(-m // c["gate_group"]) * d, "token": m}[c["gate"]]
        vecs = (2 if c["kind"] == "layer" else 1) * (2 if c["post"] else 1) * d
        return {"bytes": m * d * (SIZE[c["y"]] + 2 * SIZE[c["h"]] + SIZE[c["x"]]) + 4 * gate + vecs * SIZE[c["w"]],
                "flops": 10 * m * d}
    m, v = c["m"], c["vocab"]
    return {"bytes": m * v * SIZE[c["type"]] + (m * v // 8 if c["mask"] else 0) + m * (20 + 8 * c["top"]),
            "flops": 6 * m * v}


# ------------------------------------------------------------------- inputs

def _padded(values, pitch, fill):
    """a [rows, cols] tensor whose rows are `pitch` values apart, `fill` between them"""
    full = torch.full((values.shape[0], pitch), fill, dtype=values.dtype, device=values.device)
    full[:, :values.shape[1]] = values
    return full[:, :values.shape[1]]


def _prepare_q4(c, g):
    dev, m, n, k = "cuda", c["m"], c["n"], c["k"]
    groups = -(-k // c["group"])
    x = torch.randn((m, k), generator=g, device=dev).to(TYPES[c["x"]])
    w = torch.randint(0, 256, (n, k // 2), generator=g, device=dev, dtype=torch.uint8)
    # codes spread over 16 steps around the zero: outputs of order one
    scales = ((0.5 + torch.rand((n, groups), generator=g, device=dev)) / (4.6 * math.sqrt(k))).to(TYPES[c["s"]])
    zeros = torch.randint(5, 11, (n, groups), generator=g, device=dev, dtype=torch.uint8) if c["zeros"] else None
    out = _padded(torch.empty((m, n), dtype=TYPES[c["out"]], device=dev), n + c["pad"], 0.0)
    return {"x": _padded(x, k + c["pad"], float("nan")), "w": w, "scales": scales, "zeros": zeros, "out": out}


def _prepare_norm(c, g):
    dev, m, d = "cuda", c["m"], c["dim"]

    def rand(shape, spread, mean, t):
        return (torch.randn(shape, generator=g, device=dev) * spread + mean).to(TYPES[t])

    st = {"y": rand((m, d), 0.3, 0.02, c["y"]), "h": rand((m, d), 2.0, 0.1, c["h"]), "w1": rand((d,), 0.2, 1.0, c["w"])}
    st["w2"] = rand((d,), 0.2, 1.0, c["w"]) if c["post"] else None
    layer = c["kind"] == "layer"
    st["b1"] = rand((d,), 0.1, 0.0, c["w"]) if layer else None
    st["b2"] = rand((d,), 0.1, 0.0, c["w"]) if layer and c["post"] else None
    gate_shape = {"none": None, "channel": (1, d), "row": (-(-m // c["gate_group"]), d), "token": (m,)}[c["gate"]]
    st["gate"] = rand(gate_shape, 0.1, 0.5, "f32") if gate_shape else None
    st["h_out"] = torch.empty((m, d), dtype=TYPES[c["h"]], device=dev)
    st["x_out"] = torch.empty((m, d), dtype=TYPES[c["x"]], device=dev)
    return st


def _prepare_logprob(c, g):
    dev, m, v = "cuda", c["m"], c["vocab"]
    # a broad body, and a few tokens per row far above it
    logits = torch.randn((m, v), generator=g, device=dev) * 2.0
    peaks = torch.randint(0, v, (m, 8), generator=g, device=dev)
    logits.scatter_add_(1, peaks, 6.0 + 4.0 * torch.rand((m, 8), generator=g, device=dev))
    target = torch.randint(0, v, (m,), generator=g, device=dev)
    likely = torch.rand((m,), generator=g, device=dev) < 0.7
    target = torch.where(likely, peaks[:, 0], target)
    none = torch.rand((m,), generator=g, device=dev) < 0.02      # positions that are not scored
    target = torch.where(none, torch.full_like(target, -1), target).to(torch.int32)
    allowed = None
    if c["mask"]:
        words = -(-v // 32)
        allowed = torch.randint(-(1 << 31), 1 << 31, (m, words), generator=g, device=dev, dtype=torch.int64)
        if m > 1:
            allowed[m // 2] = 0                                  # a dead end of the grammar: nothing is allowed
        allowed = allowed.to(torch.int32)
        bits = _bits(allowed, v)
        bad = torch.rand((m, v), generator=g, device=dev) < 0.001
        logits.masked_fill_(bad & ~bits, float("nan"))           # what lies under the mask may be anything
    logits = _padded(logits.to(TYPES[c["type"]]), v + c["pad"], float("nan"))
    st = {"logits": logits, "target": target, "allowed": allowed}
    for name in ("logprob", "lse", "entropy"):
        st[name] = torch.empty((m,), dtype=torch.float32, device=dev)
    st["rank"] = torch.empty((m,), dtype=torch.int32, device=dev)
    st["top_logprob"] = torch.empty((m, c["top"]), dtype=torch.float32, device=dev)
    st["top_id"] = torch.empty((m, c["top"]), dtype=torch.int32, device=dev)
    return st


PREPARE = {"q4": _prepare_q4, "norm": _prepare_norm, "logprob": _prepare_logprob}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 17)
    st = PREPARE[case["op"]](case, g)
    st["case"] = dict(case)
    if own:
        import quantized_mixture_experts_router_gb300 as Q
        t = {"f32": Q.MOE_T_F32, "bf16": Q.MOE_T_BF16, "f16": Q.MOE_T_F16}
        st["Q"] = Q
        if case["op"] == "q4":
            st["cfg"] = Q.make_q4_cfg(case["n"], case["k"], case["group"], t[case["x"]], t[case["s"]], t[case["out"]],
                                      max_tokens=case["m"])
            st["ws"] = torch.empty(Q.moe_v41_q4_workspace_bytes(st["cfg"]), dtype=torch.uint8, device="cuda")
            Q.moe_v41_workspace_init(st["ws"])
        elif case["op"] == "norm":
            kind = {"rms": Q.MOE_NORM_RMS, "layer": Q.MOE_NORM_LAYER}[case["kind"]]
            gate = {"none": Q.MOE_GATE_NONE, "channel": Q.MOE_GATE_ROW, "row": Q.MOE_GATE_ROW,
                    "token": Q.MOE_GATE_TOKEN}[case["gate"]]
            group = {"channel": max(case["m"], 1), "row": case["gate_group"]}.get(case["gate"], 1)
            st["cfg"] = Q.make_norm_cfg(case["dim"], post_kind=kind if case["post"] else Q.MOE_NORM_NONE, pre_kind=kind,
                                        y_type=t[case["y"]], h_type=t[case["h"]], x_type=t[case["x"]],
                                        w_type=t[case["w"]], gate_kind=gate, gate_type=Q.MOE_T_F32, gate_group=group,
                                        eps=1e-6, residual_scale=0.9, block_scale=1.1)
        else:
            st["cfg"] = Q.make_logprob_cfg(case["vocab"], t[case["type"]], case["top"], case["temp"])
    return st


# --------------------------------------------------------- one pass, own calls

def _own(st):
    Q, c, cfg = st["Q"], st["case"], st["cfg"]
    if c["op"] == "q4":
        Q.moe_v41_q4_linear(cfg, st["x"], c["m"], st["x"].stride(0), st["w"], st["scales"], st["zeros"], st["out"],
                            st["out"].stride(0), st["ws"])
        return {"out": st["out"]}
    if c["op"] == "norm":
        d = c["dim"]
        Q.moe_v41_block_norm(cfg, c["m"], st["y"], d, st["w2"], st["b2"], st["gate"], d, st["h"], d, st["h_out"], d,
                             st["w1"], st["b1"], st["x_out"], d)
        return {"h": st["h_out"], "x": st["x_out"]}
    allowed = st["allowed"]
    Q.moe_v41_token_logprobs(cfg, st["logits"], c["m"], st["logits"].stride(0), allowed,
                             0 if allowed is None else allowed.stride(0), st["target"], st["logprob"], st["rank"],
                             st["lse"], st["entropy"], st["top_logprob"], st["top_id"])
    return {k: st[k] for k in ("logprob", "rank", "lse", "entropy", "top_logprob", "top_id")}


# --------------------------------------------------------- one pass, plain torch

def _codes(w):
    return torch.stack((w & 15, w >> 4), dim=-1).reshape(w.shape[0], -1)


def _bits(words, v):
    shifts = torch.arange(32, device=words.device, dtype=torch.int32)
    return (((words.unsqueeze(-1) >> shifts) & 1) != 0).reshape(words.shape[0], -1)[:, :v]


def _plain_q4(st):
    c = st["case"]
    k, group = c["k"], c["group"]
    q = _codes(st["w"]).float()
    z = st["zeros"].float().repeat_interleave(group, dim=1)[:, :k] if c["zeros"] else 8.0
    w = (q - z) * st["scales"].float().repeat_interleave(group, dim=1)[:, :k]
    return {"out": (st["x"].float() @ w.t()).to(TYPES[c["out"]])}


def _plain_normed(v, kind, w, b):
    if kind == "layer":
        v = v - v.mean(dim=-1, keepdim=True)
    v = v * torch.rsqrt((v * v).mean(dim=-1, keepdim=True) + 1e-6) * w.float()
    return v + b.float() if b is not None else v


def _plain_norm(st):
    c = st["case"]
    y = st["y"].float()
    if c["post"]:
        y = _plain_normed(y, c["kind"], st["w2"], st["b2"])
    gate = st["gate"]
    if c["gate"] == "token":
        gate = gate[:, None]
    elif c["gate"] == "row":
        gate = gate.repeat_interleave(c["gate_group"], dim=0)[:c["m"]]
    y = y if gate is None else y * gate
    h = 0.9 * st["h"].float() + 1.1 * y
    x = _plain_normed(h, c["kind"], st["w1"], st["b1"])
    return {"h": h.to(TYPES[c["h"]]), "x": x.to(TYPES[c["x"]])}


def _plain_logprob(st):
    c = st["case"]
    m, v, k = c["m"], c["vocab"], c["top"]
    low = float("-inf")
    z = st["logits"].float()
    ok = None
    if c["mask"]:
        ok = _bits(st["allowed"], v)
        z = z.masked_fill(~ok, low)
    top, ids = torch.sort(z, dim=-1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k].to(torch.int32)
    if c["mask"] and k:
        few = ok.sum(dim=-1, keepdim=True) <= torch.arange(k, device=z.device)
        ids = ids.masked_fill(few, -1)
    t = st["target"].long()
    given = t >= 0
    zt = z.gather(1, t.clamp(min=0)[:, None])
    rank = ((z > zt).sum(dim=-1) + 1).masked_fill(~given, 0).to(torch.int32)
    z = z / c["temp"]
    zmax = z.max(dim=-1, keepdim=True).values
    empty = zmax == low
    d = z - zmax.masked_fill(empty, 0.0)
    e = d.exp()
    s = e.sum(dim=-1, keepdim=True)
    lse = zmax + s.log().masked_fill(empty, 0.0)
    ent = s.log() - (e * d.masked_fill(d == low, 0.0)).sum(dim=-1, keepdim=True) / s
    lp = (zt / c["temp"] - lse).masked_fill(empty, low)
    top_lp = (top / c["temp"] - lse).masked_fill(empty, low) if k else top
    return {"logprob": lp[:, 0].masked_fill(~given, 0.0), "rank": rank, "lse": lse[:, 0],
            "entropy": ent.masked_fill(empty, 0.0)[:, 0], "top_logprob": top_lp, "top_id": ids}


PLAIN = {"q4": _plain_q4, "norm": _plain_norm, "logprob": _plain_logprob}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# --------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "q4":
        m, n, k, group = case["m"], case["n"], case["k"], case["group"]
        x = st["x"].to(f64)
        out = torch.empty((m, n), dtype=f64, device="cuda")
        step = 4096
        for r in range(0, n, step):
            w8 = st["w"][r:r + step]
            w = torch.empty((w8.shape[0], k), dtype=f64, device="cuda")
            w[:, 0::2] = w8.remainder(16).to(f64)
            w[:, 1::2] = w8.div(16, rounding_mode="floor").to(f64)
            for j in range(-(-k // group)):
                part = w[:, j * group:(j + 1) * group]
                zero = st["zeros"][r:r + step, j:j + 1].to(f64) if case["zeros"] else 8.0
                part.sub_(zero).mul_(st["scales"][r:r + step, j:j + 1].to(f64))
            out[:, r:r + step] = torch.einsum("mk,nk->mn", x, w)
        return {"out": out}
    if case["op"] == "norm":
        m, d = case["m"], case["dim"]

        def normed(v, w, b):
            mean = v.sum(1, keepdim=True) / d if case["kind"] == "layer" else 0.0
            var = ((v - mean) ** 2).sum(1, keepdim=True) / d
            r = (v - mean) / (var + 1e-6).sqrt() * w.to(f64)
            return r if b is None else r + b.to(f64)

        y = st["y"].to(f64)
        if case["post"]:
            y = normed(y, st["w2"], st["b2"])
        if case["gate"] == "token":
            y = y * st["gate"].to(f64).reshape(m, 1)
        elif case["gate"] == "channel":
            y = y * st["gate"].to(f64)
        elif case["gate"] == "row":
            y = y * st["gate"].to(f64)[torch.arange(m, device="cuda") // case["gate_group"]]
        h = st["h"].to(f64) * 0.9 + y * 1.1
        return {"h": h, "x": normed(h, st["w1"], st["b1"])}
    m, v, k, temp = case["m"], case["vocab"], case["top"], case["temp"]
    outs = {"logprob": [], "rank": [], "lse": [], "entropy": [], "top_logprob": [], "top_id": []}
    targets = st["target"].tolist()
    inf = float("inf")
    at = torch.arange(v, device="cuda")
    for t in range(m):                                            # a row at a time, over its allowed entries alone
        row = st["logits"][t]
        ids = at
        if case["mask"]:
            word = st["allowed"][t][at // 32].long()
            ids = at[((word >> (at % 32)) & 1) == 1]
        zr = row[ids].to(f64)
        z = zr / temp
        live = zr.numel() > 0
        lse = torch.logsumexp(z, 0) if live else torch.tensor(-inf, dtype=f64, device="cuda")
        p = (z - lse).exp()
        outs["lse"].append(lse)
        outs["entropy"].append((p * (lse - z)).sum() if live else torch.zeros((), dtype=f64, device="cuda"))
        if targets[t] < 0:
            outs["logprob"].append(torch.zeros((), dtype=f64, device="cuda"))
            outs["rank"].append(torch.zeros((), dtype=torch.int32, device="cuda"))
        else:
            hit = ids == targets[t]
            zt = torch.where(hit, zr, torch.full_like(zr, -inf)).max() if live else lse
            outs["logprob"].append(zt / temp - lse if live else lse)
            outs["rank"].append(((zr > zt).sum() + 1).to(torch.int32))
        n = min(k, zr.numel())
        best = torch.full((k,), -inf, dtype=f64, device="cuda")
        who = torch.full((k,), -1, dtype=torch.int32, device="cuda")
        if n:
            val = zr.topk(n).values
            # at least the n largest, ties of the n-th among them, in id order; then a stable sort keeps the lowest ids
            some = (zr >= val[-1]).nonzero()[:, 0]
            order = torch.sort(zr[some], descending=True, stable=True).indices[:n]
            best[:n] = val / temp - lse
            who[:n] = ids[some[order]].to(torch.int32)
        outs["top_logprob"].append(best)
        outs["top_id"].append(who)
    return {name: torch.stack(rows) for name, rows in outs.items()}

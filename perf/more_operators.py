"""The operators of an attention block over a paged cache, as they are measured:
rotary positions, appending keys and values with the rotation on the way, and
the attention of new tokens over the cache (single tokens, chunks, prompts).

listed() and draw() give the cases, prepare() the inputs of one, run() one
pass: in plain torch operations, or (own) through the library's calls.
"""
from __future__ import annotations

import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------- cases

def _rope(name, m, heads, dim, rot, first=0, layout="half", t="bf16", scaling="none", inverse=False, far=4000):
    """x [m, heads, dim], values first .. first + rot - 1 of each head rotated; positions below `far`"""
    c = {"op": "rope", "m": m, "heads": heads, "dim": dim, "rot": rot, "first": first, "layout": layout, "type": t,
         "scaling": scaling, "inverse": inverse, "far": far}
    return {"name": name, **c} if name else c


def _batch(batch, new, ragged, lo, hi, mix, heads, kv_heads, dim, page, order, t):
    """`batch` sequences of `new` new tokens (up to that many when ragged), lo .. hi tokens each with them"""
    return {"batch": batch, "new": new, "ragged": ragged, "lo": lo, "hi": hi, "mix": mix, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "order": order, "type": t}


def _append(name, batch, new, ragged, lo, hi, mix, heads, kv_heads, dim, page, order, t, rot, layout, x="bf16",
            scaling="none"):
    c = {"op": "append", **_batch(batch, new, ragged, lo, hi, mix, heads, kv_heads, dim, page, order, t), "rot": rot,
         "first": 0, "layout": layout, "x": x, "scaling": scaling}
    return {"name": name, **c} if name else c


def _attn(name, batch, new, ragged, lo, hi, mix, heads, kv_heads, dim, page, order, t, causal=True, window=0, tail=0):
    """tail: rows of q and out behind the last sequence"""
    c = {"op": "attn", **_batch(batch, new, ragged, lo, hi, mix, heads, kv_heads, dim, page, order, t),
         "causal": causal, "window": window, "tail": tail}
    return {"name": name, **c} if name else c


def listed():
    return [
        # the query of one decode token: latency counts
        _rope("rope_m1", 1, 32, 128, 128, far=100000),
        # the gradient of a training step's queries, the last 64 of 192 values rotated in neighbouring pairs, f32
        _rope("rope_grad_m4096", 4096, 16, 192, 64, first=128, layout="interleaved", t="f32", scaling="parts",
              inverse=True, far=30000),
        # a decode step of 48 sequences: one token each
        _append("append_m48", 48, 1, False, 10, 2000, 1, 32, 8, 128, 16, "nhd", "bf16", 128, "half"),
        # a chunk of prompts, f32 projections, part of an odd head rotated, scaled for long contexts
        _append("append_m4096", 3, 2000, True, 1, 9000, 2, 20, 5, 80, 64, "hnd", "f16", 64, "interleaved", x="f32",
                scaling="parts"),
        # one decode token in a short context: latency counts
        _attn("decode_b1", 1, 1, False, 700, 700, 3, 32, 8, 128, 16, "nhd", "bf16"),
        # one decode token in a long context
        _attn("decode_b1_long", 1, 1, False, 131000, 131000, 4, 64, 8, 128, 64, "nhd", "bf16"),
        # a decode batch of every length, padded as a captured step is
        _attn("decode_b60", 60, 1, False, 40, 8000, 5, 40, 8, 128, 32, "hnd", "f16", tail=4),
        # five drafted tokens of each sequence, checked at once
        _attn("verify_b16", 16, 5, False, 3000, 9000, 6, 64, 8, 128, 16, "nhd", "bf16"),
        # the next chunk of a long prompt
        _attn("chunk_m2048", 1, 2048, False, 10000, 10000, 7, 32, 8, 128, 64, "nhd", "bf16"),
        # prompts of every length, a head of 96 values, one key head a query head
        _attn("prompts_b7", 7, 2500, True, 1, 1, 8, 16, 16, 96, 128, "hnd", "f16"),
        # a chunk and others beside it in a window of 1000 tokens
        _attn("window_b3", 3, 1024, True, 5000, 30000, 9, 24, 4, 128, 32, "nhd", "bf16", window=1000),
        # decoder tokens against an encoder's states of another length
        _attn("cross_b4", 4, 448, True, 200, 1500, 10, 16, 16, 64, 8, "hnd", "bf16", causal=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lengths(c):
    """new tokens and all tokens of each sequence"""
    rng = random.Random(c["mix"])
    new, kv = [], []
    for _ in range(c["batch"]):
        n = rng.randint(1, c["new"]) if c["ragged"] else c["new"]
        k = _log(rng, c["lo"], c["hi"])
        new.append(n)
        kv.append(k if c["op"] == "attn" and not c["causal"] else max(n, k))
    if c["ragged"] and c["batch"] > 4:
        new[c["batch"] // 2] = 0                                 # a sequence that waits
    if c["ragged"]:
        new[0] = c["new"]
        kv[0] = max(kv[0], new[0]) if c["op"] != "attn" or c["causal"] else kv[0]
    return new, kv


def draw(rng):
    while True:
        c = _draw(rng)
        w = work(c)
        # as costly as the largest listed ones at the most
        if w["bytes"] <= 5.3e8 and w["flops"] <= 2.9e11:
            return c


def _draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn", "attn", "attn"])
    t = rng.choice(["bf16", "f16"])
    dim = rng.choice([64, 80, 96, 128, 128])
    rot = rng.choice([dim, dim, dim // 2])
    layout = rng.choice(["half", "interleaved"])
    scaling = rng.choice(["none", "linear", "ntk", "parts"])
    if op == "rope":
        dim = rng.choice([64, 96, 128, 192])
        rot = rng.choice([dim, dim // 2, 32])
        return _rope(None, _log(rng, 1, 4096), rng.randint(1, 40), dim, rot, rng.choice([0, dim - rot]), layout,
                     rng.choice(["f32", "bf16", "f16"]), scaling, rng.random() < 0.4, rng.choice([4000, 100000]))
    kv_heads = rng.randint(1, 8)
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 8, 16])
    page = 8 << rng.randint(0, 5)
    order = rng.choice(["nhd", "hnd"])
    mix = rng.randint(0, 10 ** 6)
    if op == "append":
        new = rng.choice([1, 1, _log(rng, 2, 2000)])
        return _append(None, rng.randint(1, 64 if new == 1 else 4), new, new > 1 and rng.random() < 0.7, 1, 5000, mix,
                       kv_heads * group, kv_heads, dim, page, order, t, rot, layout, rng.choice(["f32", t]), scaling)
    kind = rng.choice(["decode", "decode", "verify", "chunk", "prompts", "window", "cross"])
    heads = kv_heads * group
    tail = rng.choice([0, 0, 3])
    if kind == "decode":
        lo = _log(rng, 20, 20000)
        return _attn(None, _log(rng, 1, 64), 1, False, lo, lo * rng.choice([1, 4]), mix, heads, kv_heads, dim, page,
                     order, t, tail=tail)
    if kind == "verify":
        return _attn(None, rng.randint(1, 16), rng.randint(2, 9), False, 100, _log(rng, 200, 10000), mix, heads,
                     kv_heads, dim, page, order, t, tail=tail)
    if kind == "chunk":
        return _attn(None, rng.randint(1, 2), _log(rng, 33, 2048), False, 500, _log(rng, 1000, 12000), mix, heads,
                     kv_heads, dim, page, order, t, tail=tail)
    if kind == "prompts":
        return _attn(None, rng.randint(1, 7), _log(rng, 33, 2500), True, 1, 1, mix, heads, kv_heads, dim, page, order,
                     t, tail=tail)
    if kind == "window":
        return _attn(None, rng.randint(1, 4), _log(rng, 1, 1024), rng.random() < 0.5, 2000, 20000, mix, heads,
                     kv_heads, dim, page, order, t, window=_log(rng, 30, 2000), tail=tail)
    return _attn(None, rng.randint(1, 4), _log(rng, 1, 448), True, 100, 1500, mix, heads, kv_heads, dim, page, order,
                 t, causal=False, tail=tail)


def work(c):
    if c["op"] == "rope":
        values = c["m"] * c["heads"] * c["dim"]
        return {"bytes": 2 * values * SIZE[c["type"]] + 4 * c["m"] + 4 * c["rot"],
                "flops": 3 * c["m"] * c["heads"] * c["rot"]}
    new, kv = _lengths(c)
    m, d = sum(new), c["dim"]
    if c["op"] == "append":
        values = m * d * (c["heads"] + 2 * c["kv_heads"])
        return {"bytes": values * (SIZE[c["x"]] + SIZE[c["type"]]) + 12 * c["batch"] + 4 * c["rot"],
                "flops": 3 * m * c["rot"] * (c["heads"] + c["kv_heads"])}
    pairs = keys = 0
    for n, length in zip(new, kv):
        if not n:
            continue
        if not c["causal"]:
            pairs += n * length
            keys += length
            continue
        first = length - n                                       # the first new token's position
        if c["window"]:
            pairs += sum(min(p + 1, c["window"]) for p in range(first, length))
            keys += length - max(0, first - c["window"] + 1)
        else:
            pairs += n * first + n * (n + 1) // 2
            keys += length
    return {"bytes": keys * c["kv_heads"] * d * 2 * SIZE[c["type"]] + m * c["heads"] * (
        2 * d * SIZE[c["type"]] + 4) + keys // c["page"] * 4 + 12 * c["batch"],
        "flops": 4 * d * c["heads"] * pairs}


# ------------------------------------------------------------------- inputs

BASE, FACTOR, TRAINED = 500000.0, 8.0, 4096                      # of the rotation; a context stretched eight times


def _freqs(rot, scaling):
    """angle per position of each pair, and the factor of the rotated values"""
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    f = BASE ** (-i / rot)
    if scaling == "linear":
        return f / FACTOR, 1.0
    if scaling == "ntk":
        return (BASE * FACTOR ** (rot / (rot - 2))) ** (-i / rot), 1.0
    if scaling == "parts":                                       # slow pairs are stretched, fast ones kept
        turns = TRAINED * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        return f / FACTOR * (1 - keep) + f * keep, 0.1 * math.log(FACTOR) + 1.0
    return f, 1.0


def _table(c, new, kv, g):
    """pages in any order, -1 where a sequence has none; and how many there are"""
    page = c["page"]
    need = [-(-k // page) for k in kv]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((c["batch"], max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, n_pages


def _cache(c, n_pages, fill):
    """[n_pages, page, kv_heads, dim] in memory, or [n_pages, kv_heads, page, dim], seen as the first"""
    shape = (n_pages, c["page"], c["kv_heads"], c["dim"])
    if c["order"] == "hnd":
        return fill((shape[0], shape[2], shape[1], shape[3])).transpose(1, 2)
    return fill(shape)


def _prepare_rope(c, g):
    t, shape = TYPES[c["type"]], (c["m"], c["heads"], c["dim"])
    f, mag = _freqs(c["rot"], c["scaling"])
    return {"x": torch.randn(shape, generator=g, device="cuda").to(t), "freqs": f.cuda(), "magnitude": mag,
            "pos": torch.randint(0, c["far"], (c["m"],), generator=g, device="cuda", dtype=torch.int32),
            "out": torch.empty(shape, dtype=t, device="cuda")}


def _sequences(c, g):
    new, kv = _lengths(c)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    table, n_pages = _table(c, new, kv, g)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    return {"new": new, "kv": kv, "cu": cu, "cu_new": ints(cu), "kv_len": ints(kv), "table": table,
            "n_pages": n_pages}


def _prepare_append(c, g):
    st = _sequences(c, g)
    m, d, t, x = st["cu"][-1], c["dim"], TYPES[c["type"]], TYPES[c["x"]]
    f, mag = _freqs(c["rot"], c["scaling"])
    # queries, keys and values of a token beside each other, as one projection gives them
    qkv = torch.randn((m, c["heads"] + 2 * c["kv_heads"], d), generator=g, device="cuda").to(x)
    h, k = c["heads"], c["kv_heads"]
    st.update(freqs=f.cuda(), magnitude=mag, q=qkv[:, :h], k=qkv[:, h:h + k], v=qkv[:, h + k:],
              q_out=torch.empty((m, h, d), dtype=t, device="cuda"))
    for name in ("k_cache", "v_cache"):
        st[name] = _cache(c, st["n_pages"], lambda s: torch.randn(s, generator=g, device="cuda").to(t))
    st["status"] = torch.zeros((1,), dtype=torch.int32, device="cuda")
    return st


def _prepare_attn(c, g):
    st = _sequences(c, g)
    m, d, t = st["cu"][-1] + c["tail"], c["dim"], TYPES[c["type"]]
    # scores of a standard deviation of two: some keys stand out, none is alone
    st["q"] = (torch.randn((m, c["heads"], d), generator=g, device="cuda") * 2.0).to(t)
    for name in ("k_cache", "v_cache"):
        st[name] = _cache(c, st["n_pages"], lambda s: torch.randn(s, generator=g, device="cuda").to(t))
    # slots that no token has been written to may hold anything
    for b, length in enumerate(st["kv"]):
        if length % c["page"]:
            last = int(st["table"][b, length // c["page"]])
            for name in ("k_cache", "v_cache"):
                st[name][last, length % c["page"]:] = float("nan")
    st["out"] = torch.zeros((m, c["heads"], d), dtype=t, device="cuda")
    st["lse"] = torch.zeros((m, c["heads"]), dtype=torch.float32, device="cuda")
    return st


PREPARE = {"rope": _prepare_rope, "append": _prepare_append, "attn": _prepare_attn}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 29)
    st = PREPARE[case["op"]](case, g)
    st["case"] = dict(case)
    if own:
        _prepare_own(st)
    return st


def _prepare_own(st):
    import quantized_mixture_experts_router_gb300 as Q
    c = st["case"]
    t = {"f32": Q.MOE_T_F32, "bf16": Q.MOE_T_BF16, "f16": Q.MOE_T_F16}
    st["Q"] = Q
    if c["op"] != "attn":
        kind = {"none": Q.MOE_ROPE_SCALE_NONE, "linear": Q.MOE_ROPE_SCALE_LINEAR, "ntk": Q.MOE_ROPE_SCALE_BASE,
                "parts": Q.MOE_ROPE_SCALE_PARTS}[c["scaling"]]
        freqs, magnitude = Q.moe_v41_rope_freqs(c["rot"], BASE, kind, FACTOR, TRAINED)
        st["freqs"] = torch.tensor(freqs, dtype=torch.float64, device="cuda")
        layout = {"half": Q.MOE_ROPE_HALF, "interleaved": Q.MOE_ROPE_INTERLEAVED}[c["layout"]]
        given = t[c["x" if c["op"] == "append" else "type"]]
        st["rope"] = Q.make_rope_cfg(c["dim"], c["rot"], c["first"], layout, given,
                                     inverse=c.get("inverse", False), magnitude=magnitude)
    if c["op"] != "rope":
        k = st["k_cache"]
        st["kv_cfg"] = Q.make_kv_cfg(c["kv_heads"], c["dim"], c["page"], st["n_pages"], t[c["type"]],
                                     page_pitch=k.stride(0), token_pitch=k.stride(1), head_pitch=k.stride(2))
        st["seqs"] = Q.make_seqs(c["batch"], st["cu_new"], st["kv_len"], st["table"], st["table"].shape[1],
                                 st["table"].stride(0))
    if c["op"] == "attn":
        st["cfg"] = Q.make_attn_cfg(st["kv_cfg"], c["heads"], causal=c["causal"], window=c["window"],
                                    scale=1.0 / math.sqrt(c["dim"]))
        st["ws"] = torch.empty(Q.moe_v41_attn_workspace_bytes(st["cfg"]), dtype=torch.uint8, device="cuda")
        Q.moe_v41_workspace_init(st["ws"])


# --------------------------------------------------------- one pass, own calls

def _own(st):
    Q, c = st["Q"], st["case"]
    if c["op"] == "rope":
        x, out = st["x"], st["out"]
        Q.moe_v41_rope(st["rope"], c["m"], c["heads"], x, x.stride(0), x.stride(1), st["pos"], st["freqs"], out,
                       out.stride(0), out.stride(1))
        return out
    if c["op"] == "append":
        q, k, v, q_out = st["q"], st["k"], st["v"], st["q_out"]
        Q.moe_v41_kv_append(st["kv_cfg"], st["rope"], st["seqs"], st["cu"][-1], k, k.stride(0), v, v.stride(0),
                            st["k_cache"], st["v_cache"], c["heads"], q, q.stride(0), q_out, q_out.stride(0),
                            st["freqs"], None, st["status"])
        return {"q": q_out, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    q, out, lse = st["q"], st["out"], st["lse"]
    Q.moe_v41_paged_attention(st["cfg"], st["seqs"], q.shape[0], c["new"], q, q.stride(0), st["k_cache"],
                              st["v_cache"], out, out.stride(0), lse, lse.stride(0), st["ws"])
    return {"out": out, "lse": lse}


# --------------------------------------------------------- one pass, plain torch

def _rotated(x, pos, c, freqs, magnitude, inverse=False):
    """x [m, heads, dim] in 32 bits, the angles in 64"""
    first, rot = c["first"], c["rot"]
    a = pos.double()[:, None] * freqs
    cos, sin = (a.cos() * magnitude).float()[:, None], (a.sin() * magnitude).float()[:, None]
    if inverse:
        sin = -sin
    part = x[..., first:first + rot]
    if c["layout"] == "half":
        u, w = part[..., :rot // 2], part[..., rot // 2:]
        part = torch.cat((u * cos - w * sin, w * cos + u * sin), dim=-1)
    else:
        u, w = part[..., 0::2], part[..., 1::2]
        part = torch.stack((u * cos - w * sin, w * cos + u * sin), dim=-1).flatten(-2)
    return torch.cat((x[..., :first], part, x[..., first + rot:]), dim=-1)


def _plain_rope(st):
    c = st["case"]
    return _rotated(st["x"].float(), st["pos"], c, st["freqs"], st["magnitude"], c["inverse"]).to(st["x"].dtype)


def _plain_append(st):
    c, t = st["case"], TYPES[st["case"]["type"]]
    m = st["cu"][-1]
    tok = torch.arange(m, device="cuda", dtype=torch.int32)
    seq = (tok[:, None] >= st["cu_new"][None, 1:]).sum(dim=1)
    pos = tok - st["cu_new"][1:][seq] + st["kv_len"][seq]
    q = _rotated(st["q"].float(), pos, c, st["freqs"], st["magnitude"]).to(t)
    k = _rotated(st["k"].float(), pos, c, st["freqs"], st["magnitude"]).to(t)
    page, slot = st["table"][seq, pos // c["page"]].long(), (pos % c["page"]).long()
    st["k_cache"][page, slot] = k
    st["v_cache"][page, slot] = st["v"].to(t)
    return {"q": q, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _plain_attn(st):
    """all sequences at once, padded to the longest"""
    c = st["case"]
    h, kh, d, page, window = c["heads"], c["kv_heads"], c["dim"], c["page"], c["window"]
    group, low = h // kh, float("-inf")
    start, new = st["cu_new"][:-1].long(), st["cu_new"].diff()
    i = torch.arange(max(st["new"]), device="cuda")
    pos = (st["kv_len"] - new)[:, None] + i                        # of each sequence's new tokens
    given = i < new[:, None]
    first = (pos[:, :1] - window + 1).clamp(min=0) if window else torch.zeros_like(pos[:, :1])
    most = max(min(k, n + window - 1) if window else k for n, k in zip(st["new"], st["kv"]))
    j = first + torch.arange(most, device="cuda")                  # of the keys that any of them sees
    held = j < st["kv_len"][:, None]
    pages = st["table"].gather(1, (j // page).clamp(max=st["table"].shape[1] - 1)).clamp(min=0).long()
    k = st["k_cache"][pages, j % page].float().permute(0, 2, 3, 1)
    v = st["v_cache"][pages, j % page].float().masked_fill(~held[:, :, None, None], 0.0).transpose(1, 2)
    rows = (start[:, None] + i).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][rows].float().unflatten(2, (kh, group)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    s = (q @ k).mul_(1.0 / math.sqrt(d)).unflatten(2, (group, i.numel()))
    hidden = ~held[:, None]
    if c["causal"]:
        hidden = hidden | (j[:, None] > pos[:, :, None])
    if window:
        hidden |= j[:, None] <= pos[:, :, None] - window
    s.masked_fill_(hidden[:, None, None], low)
    top = s.amax(dim=-1, keepdim=True)
    s.sub_(top.masked_fill(top == low, 0.0)).exp_()
    total = s.sum(dim=-1, keepdim=True)
    o = (s.flatten(2, 3) @ v).unflatten(2, (group, i.numel())) / total
    out, lse = torch.zeros_like(st["out"]), torch.zeros_like(st["lse"])
    o = o.masked_fill(total == 0.0, 0.0).permute(0, 3, 1, 2, 4).flatten(2, 3)
    out[rows[given]] = o[given].to(out.dtype)
    lse[rows[given]] = (top + total.log())[..., 0].permute(0, 3, 1, 2).flatten(2, 3)[given]
    return {"out": out, "lse": lse}


PLAIN = {"rope": _plain_rope, "append": _plain_append, "attn": _plain_attn}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# --------------------------------------------------------- the definition, in 64 bits

def _turned(x, pos, c, sign):
    """every pair as a complex number, multiplied by magnitude e^(i sign pos freq)"""
    f, mag = _freqs(c["rot"], c["scaling"])
    half, first = c["rot"] // 2, c["first"]
    pair = torch.arange(half, device="cuda")
    re = first + (pair if c["layout"] == "half" else 2 * pair)
    im = first + (pair + half if c["layout"] == "half" else 2 * pair + 1)
    angle = sign * pos.to(torch.float64).reshape(-1, 1, 1) * f.cuda()
    z = torch.complex(x[..., re], x[..., im]) * torch.polar(torch.full_like(angle, mag), angle)
    y = x.clone()
    y[..., re], y[..., im] = z.real, z.imag
    return y


def exact(case, seed):
    st = prepare(case, seed)
    c, f64 = case, torch.float64
    if c["op"] == "rope":
        return _turned(st["x"].to(f64), st["pos"], c, -1.0 if c["inverse"] else 1.0)
    if c["op"] == "append":
        pos = torch.cat([torch.arange(k - n, k) for n, k in zip(st["new"], st["kv"])]).cuda()
        k, v = _turned(st["k"].to(f64), pos, c, 1.0), st["v"].to(f64)
        caches = {"k_cache": st["k_cache"].to(f64), "v_cache": st["v_cache"].to(f64)}
        for b in range(c["batch"]):
            table = st["table"][b].tolist()
            lo, hi = st["kv"][b] - st["new"][b], st["kv"][b]
            while lo < hi:                                       # a page at a time
                end = min(hi, (lo // c["page"] + 1) * c["page"])
                src = st["cu"][b] + lo - (st["kv"][b] - st["new"][b])
                at, to = lo % c["page"], (end - 1) % c["page"] + 1
                for name, given in (("k_cache", k), ("v_cache", v)):
                    caches[name][table[lo // c["page"]], at:to] = given[src:src + end - lo]
                lo = end
        return {"q": _turned(st["q"].to(f64), pos, c, 1.0), **caches}
    group, scale = c["heads"] // c["kv_heads"], float(c["dim"]) ** -0.5
    out, lse = st["out"].to(f64), st["lse"].to(f64)
    for b in range(c["batch"]):
        n, length, at = st["new"][b], st["kv"][b], st["cu"][b]
        if n == 0:
            continue
        slot = torch.arange(length, device="cuda")
        where = st["table"][b].long()[slot // c["page"]], slot % c["page"]
        pos = torch.arange(length - n, length, device="cuda").reshape(n, 1, 1)
        for h in range(c["kv_heads"]):
            k, v = st["k_cache"][where[0], where[1], h].to(f64), st["v_cache"][where[0], where[1], h].to(f64)
            q = st["q"][at:at + n, h * group:(h + 1) * group].to(f64)
            s = torch.einsum("ngd,ld->ngl", q, k) * scale
            if c["causal"]:
                hidden = slot > pos
                if c["window"]:
                    hidden = hidden | (slot + c["window"] <= pos)
                s.masked_fill_(hidden, float("-inf"))
            z = torch.logsumexp(s, dim=-1)
            s.sub_(z[..., None]).exp_()
            out[at:at + n, h * group:(h + 1) * group] = torch.einsum("ngl,ld->ngd", s, v)
            lse[at:at + n, h * group:(h + 1) * group] = z
    return {"out": out, "lse": lse}

"""Rotary positions, the paged cache and attention over it on the GPU against
plain 64-bit torch.

u is half a step of the cache's type (2^-8 bf16, 2^-11 fp16), U = 2^-24 of f32.
"""
import math

import pytest
import torch
from test_gpu_ops import INF, NAN, T, U, Q, close, code, gen, half_step, pitched  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ rotary positions

def turned(x, pos, freqs, first, layout, magnitude=1.0, inverse=False):
    """x [m, heads, dim] in 64 bits"""
    x, half = x.double().clone(), freqs.numel()
    a = pos.double()[:, None, None] * freqs * (-1.0 if inverse else 1.0)
    i = torch.arange(half, device="cuda")
    lo, hi = (first + i, first + i + half) if layout == 0 else (first + 2 * i, first + 2 * i + 1)
    s, t = x[..., lo], x[..., hi]
    x[..., lo] = (s * a.cos() - t * a.sin()) * magnitude
    x[..., hi] = (t * a.cos() + s * a.sin()) * magnitude
    return x


def rope_tol(x, pos, freqs, first, layout, magnitude, t):
    """both products of a pair, with a sine and cosine of 2 U (sincospi) + pi U (its argument's rounding; at most half a
    turn) + U (the factor), three roundings of U, and the output's own: under 10 U of the pair's sizes"""
    m = turned(x.abs(), pos * 0, freqs, first, layout)
    half = freqs.numel()
    i = torch.arange(half, device="cuda")
    lo, hi = (first + i, first + i + half) if layout == 0 else (first + 2 * i, first + 2 * i + 1)
    both = (m[..., lo] + m[..., hi]) * abs(magnitude)
    m[..., lo], m[..., hi] = both, both
    return 10 * U * m


# m, heads, dim, rot, first, layout, type, magnitude, inverse, pitches
ROPE = [
    (1, 32, 128, 128, 0, 0, "bf16", 1.0, False, 0),
    (1, 1, 2, 2, 0, 1, "f32", 1.0, False, 0),
    (7, 3, 192, 64, 128, 1, "f32", 1.2, True, 0),
    (300, 40, 128, 64, 0, 0, "f16", 1.0, False, 8),
    (33, 5, 80, 40, 40, 0, "bf16", 0.9, True, 0),       # halves of 20: one pair at a time
    (33, 5, 80, 40, 8, 1, "bf16", 1.0, False, 0),
    (19, 3, 7, 4, 2, 0, "f16", 1.0, False, 1),          # odd heads
    (19, 3, 7, 6, 1, 1, "f32", 1.0, True, 3),
    (5000, 2, 64, 64, 0, 0, "bf16", 1.0, False, 0),
    (2, 2, 1024, 1024, 0, 0, "f32", 1.0, False, 0),
    (2000, 1, 16, 0, 4, 0, "bf16", 1.0, False, 0),      # nothing to rotate: a copy
]


@pytest.mark.parametrize("c", ROPE, ids=str)
@pytest.mark.parametrize("in_place", [False, True])
def test_rope_against_64_bits(Q, c, in_place):  # noqa: F811
    m, heads, dim, rot, first, layout, t, mag, inverse, pad = c
    g = gen(m + dim)
    full, x = pitched(m, heads * dim, heads * dim + pad, T[t], 77.0)
    x.copy_(torch.randn((m, heads * dim), generator=g, device="cuda"))
    pos = torch.randint(-5, 200000, (m,), generator=g, device="cuda", dtype=torch.int32)
    pos[0] = 2 ** 31 - 1
    freqs, _ = Q.moe_v41_rope_freqs(rot, 500000.0)
    freqs = torch.tensor(freqs, dtype=torch.float64, device="cuda")
    cfg = Q.make_rope_cfg(dim, rot, first, layout, code(Q, t), inverse, mag)
    x3 = x.clone().view(m, heads, dim)
    mag = torch.tensor(mag).item()                                # the f32 that the call is given
    want = turned(x3, pos, freqs, first, layout, mag, inverse)
    tol = rope_tol(x3, pos, freqs, first, layout, mag, t) + half_step(t, want) * 1.001
    # angles of up to 2^31 radians in 64 bits: 2^-20 of a radian here and there
    tol[0] += 2.0 ** -20 * x3[0].double().abs().max()
    if in_place:
        out = x
    else:
        out = torch.full((m, heads * dim + 8), 5.0, dtype=T[t], device="cuda")[:, :heads * dim]
    Q.moe_v41_rope(cfg, m, heads, x, x.stride(0), dim, pos, freqs, out, out.stride(0), dim)
    close(out.reshape(m, heads, dim).double(), want, tol, "rope")
    keep = torch.ones(dim, dtype=torch.bool, device="cuda")
    keep[first:first + rot] = False
    assert torch.equal(out.reshape(m, heads, dim)[..., keep], x3[..., keep])
    if pad:
        assert (full[:, heads * dim:] == 77.0).all()
    if not in_place:
        assert torch.equal(x.reshape(m, heads, dim), x3)


def test_rope_heads_first(Q):  # noqa: F811
    """[heads, m, dim] in memory, as a training step may hold it, into [m, heads, dim]"""
    m, heads, dim = 37, 6, 64
    x = torch.randn((heads, m, dim), generator=gen(1), device="cuda")
    pos = torch.arange(m, device="cuda", dtype=torch.int32)
    f, _ = Q.moe_v41_rope_freqs(dim)
    f = torch.tensor(f, dtype=torch.float64, device="cuda")
    out = torch.empty((m, heads, dim), device="cuda")
    Q.moe_v41_rope(Q.make_rope_cfg(dim, x_type=Q.MOE_T_F32), m, heads, x, dim, m * dim, pos, f, out, heads * dim, dim)
    xs = x.transpose(0, 1)
    close(out, turned(xs, pos, f, 0, 0), rope_tol(xs, pos, f, 0, 0, 1.0, "f32") + U * 4, "rope")


@pytest.mark.parametrize("layout", [0, 1])
def test_rope_inverse_is_the_gradient(Q, layout):  # noqa: F811
    """of sum(w * rope(x)) by differences: the map is linear, so a difference over any step is exact but for rounding"""
    m, heads, dim, rot, first = 5, 2, 24, 16, 8
    g = gen(4)
    x, w = (torch.randn((m, heads, dim), generator=g, device="cuda") for _ in range(2))
    pos = torch.tensor([0, 1, 17, 5000, 130000], dtype=torch.int32, device="cuda")
    f, _ = Q.moe_v41_rope_freqs(rot, 10000.0)
    f = torch.tensor(f, dtype=torch.float64, device="cuda")

    def rope(v, inverse):
        out = torch.empty_like(v)
        Q.moe_v41_rope(Q.make_rope_cfg(dim, rot, first, layout, Q.MOE_T_F32, inverse, 1.25), m, heads, v,
                       heads * dim, dim, pos, f, out, heads * dim, dim)
        return out

    grad = rope(w, True)
    for k in range(dim):
        step = torch.zeros_like(x)
        step[..., k] = 1.0
        change = ((rope(x + step, False).double() - rope(x, False).double()) * w.double()).sum(-1)
        # two outputs of 10 U of |x| + 1 sizes each, three of them under the weights, and x + 1's own rounding
        tol = 40 * U * 1.25 * ((x.abs().amax(-1) + 1) * w.abs().sum(-1)).double()
        close(grad[..., k].double(), change, tol, f"gradient of value {k}")


# ------------------------------------------------------------------ a paged cache and its sequences

class Cache:
    def __init__(self, Q, new, kv, heads, kv_heads, dim, page=16, t="bf16", order="nhd", tail=0, seed=0, fill="rand",
                 extra_pages=3, pad=0):
        g = self.g = gen(seed)
        self.Q, self.new, self.kv, self.heads, self.kv_heads, self.dim = Q, new, kv, heads, kv_heads, dim
        self.page, self.t, self.batch, self.tail = page, t, len(new), tail
        self.cu = [0]
        for n in new:
            self.cu.append(self.cu[-1] + n)
        self.m = self.cu[-1] + tail
        need = [-(-max(k, 0) // page) for k in kv]
        self.n_pages = sum(need) + extra_pages
        perm = torch.randperm(self.n_pages, generator=g, device="cuda").to(torch.int32)
        self.cols = max(max(need), 1)
        self.table = torch.full((self.batch, self.cols + 2), -7, dtype=torch.int32, device="cuda")[:, :self.cols]
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        shape = (self.n_pages, page, kv_heads, dim)
        self.caches = []
        for _ in range(2):
            if order == "hnd":
                c = torch.empty((shape[0], kv_heads, page, dim + pad), dtype=T[t], device="cuda")[..., :dim].transpose(1, 2)
            else:
                c = torch.empty((shape[0], page, kv_heads, dim + pad), dtype=T[t], device="cuda")[..., :dim]
            c.copy_(torch.randn(shape, generator=g, device="cuda"))
            self.caches.append(c)
        self.k, self.v = self.caches
        self.ints = [torch.tensor(a, dtype=torch.int32, device="cuda") for a in (self.cu, kv)]
        self.seqs = Q.make_seqs(self.batch, *self.ints, self.table, self.cols, self.table.stride(0))
        s = self.k.stride()
        self.kv_cfg = Q.make_kv_cfg(kv_heads, dim, page, self.n_pages, code(Q, t), s[0], s[1], s[2])

    def positions(self):
        return torch.cat([torch.arange(k - n, k) for n, k in zip(self.new, self.kv)] + [torch.empty(0)]).long().cuda()

    def slots(self, b, length=None):
        j = torch.arange(self.kv[b] if length is None else length, device="cuda")
        return self.table[b].long()[j // self.page], j % self.page

    def spoil(self, value):
        """every slot that holds no token of a sequence"""
        held = torch.zeros((self.n_pages, self.page), dtype=torch.bool, device="cuda")
        for b in range(self.batch):
            held[self.slots(b)] = True
        for c in self.caches:
            c[~held] = value


class Attn(Cache):
    def __init__(self, Q, *a, causal=True, window=0, scale=None, spread=2.0, padq=0, max_new=None, **kw):
        super().__init__(Q, *a, **kw)
        self.causal, self.window = causal, window
        self.scale = torch.tensor(self.dim ** -0.5 if scale is None else scale, dtype=torch.float32).item()
        row = self.heads * self.dim
        _, q = pitched(self.m, row, row + padq, T[self.t], NAN)
        q.copy_(torch.randn((self.m, row), generator=self.g, device="cuda") * spread)
        q[self.cu[-1]:] = NAN
        self.q = q
        self.full, self.out = pitched(self.m, row, row + padq, T[self.t], 77.0)
        self.lse = torch.full((self.m, self.heads), 77.0, device="cuda")
        self.cfg = Q.make_attn_cfg(self.kv_cfg, self.heads, causal, window, self.scale)
        self.max_new = max(self.new) if max_new is None else max_new
        self.ws = torch.empty(Q.moe_v41_attn_workspace_bytes(self.cfg), dtype=torch.uint8, device="cuda")
        Q.moe_v41_workspace_init(self.ws)

    def call(self, stream=None, lse=True):
        self.Q.moe_v41_paged_attention(self.cfg, self.seqs, self.m, self.max_new, self.q, self.q.stride(0), self.k,
                                       self.v, self.out, self.out.stride(0), self.lse if lse else None, self.heads,
                                       self.ws, stream=stream)

    def visible(self, b):
        n, length = self.new[b], self.kv[b]
        p = torch.arange(length - n, length, device="cuda")[:, None]
        j = torch.arange(length, device="cuda")[None]
        ok = torch.ones((n, length), dtype=torch.bool, device="cuda")
        if self.causal:
            ok = j <= p
        if self.window:
            ok = ok & (j > p - self.window)
        return ok

    def check(self, only=None):
        u = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}[self.t]
        group = self.heads // self.kv_heads
        out = self.out.view(self.m, self.heads, self.dim) if self.out.is_contiguous() else \
            self.out.unflatten(1, (self.heads, self.dim))
        for b in range(self.batch) if only is None else only:
            n, length, at = self.new[b], max(self.kv[b], 0), self.cu[b]
            if length == 0:
                assert (self.out[at:at + n] == 0).all() and (self.lse[at:at + n] == -INF).all()
            if n == 0 or length == 0:
                continue
            where, ok = self.slots(b), self.visible(b)
            for h in range(self.kv_heads):
                k, v = self.k[where[0], where[1], h].double(), self.v[where[0], where[1], h].double()
                q = self.q[at:at + n].unflatten(1, (self.heads, self.dim))[:, h * group:(h + 1) * group].double()
                s = torch.einsum("ngd,ld->ngl", q, k) * self.scale
                s = s.masked_fill(~ok[:, None], -INF)
                some = ok.any(1)
                z = torch.logsumexp(s, -1)
                p = torch.where(some[:, None, None], (s - z[..., None]).exp(), 0.0)
                want = p @ v
                big = torch.einsum("ngl,ld->ngd", p, v.abs())
                # scores: head_dim products in f32, cut or rounded at 2 U each; the exponential: its argument's rounding
                # (U of the score in bits, twice) and 2^-22 of its own
                size = (q.abs().amax(-1) * k.abs().sum(-1).max() * self.scale)[..., None]
                top = s.masked_fill(~ok[:, None], 0.0).abs().amax(-1, keepdim=True)
                e = 2 * U * (self.dim + 8) * size + 8 * U * top + 2.0 ** -20
                # weights rounded to the cache's type (fp16: to 2^-31 of the largest at the least), sums of f32
                tol = (u + 2 * e + 2 * U * (length / 16 + 64)) * big + half_step(self.t, want) * 1.01 + 2.0 ** -31 * length
                got = out[at:at + n, h * group:(h + 1) * group].double()
                close(got, want, tol, f"out of sequence {b}, key head {h}")
                # roundings of random sign: well under half a step of the weights and of the output in norm
                assert (got - want).norm() <= (0.6 * u * 2 ** 0.5 + 4e-6) * max(float(want.norm()), float(big.norm())) + 1e-30
                lse = self.lse[at:at + n, h * group:(h + 1) * group].double()
                gap = torch.where(some[:, None], lse - z, 0.0).abs()
                assert (gap <= e[..., 0] + 2 * U * (length / 16 + 64) + 4 * U * (z.abs().nan_to_num(0, 0, 0) + 8)).all()
                assert (lse[~some] == -INF).all() and (got[~some] == 0).all()
        if self.tail:
            assert (self.out[self.cu[-1]:] == 77.0).all() and (self.lse[self.cu[-1]:] == 77.0).all()
        if self.full.shape[1] > self.heads * self.dim:
            assert (self.full[:, self.heads * self.dim:] == 77.0).all()
        assert self.Q.moe_v41_read_status(self.ws) == 0


def desc(c):
    return "-".join(f"{k}{v}" for k, v in c.items()).replace(" ", "")


# single tokens and a few of them
FEW = [
    dict(new=[1], kv=[1], heads=1, kv_heads=1, dim=16, page=8),
    dict(new=[1], kv=[700], heads=32, kv_heads=8, dim=128, page=16),
    dict(new=[1], kv=[33], heads=4, kv_heads=1, dim=128, page=8),
    dict(new=[1], kv=[20000], heads=16, kv_heads=1, dim=128, page=64),
    dict(new=[1, 1, 1], kv=[5, 4097, 32], heads=6, kv_heads=2, dim=64, page=32, t="f16", order="hnd"),
    dict(new=[1] * 40, kv=list(range(1, 2000, 50)), heads=10, kv_heads=2, dim=80, page=16, tail=3, padq=8),
    dict(new=[1] * 300, kv=[(7 * i) % 200 + 1 for i in range(300)], heads=4, kv_heads=4, dim=96, page=8, t="f16"),
    dict(new=[1, 0, 1, 0, 0, 1], kv=[0, 50, 9, 0, 3, 129], heads=5, kv_heads=1, dim=24, page=8, tail=1),
    dict(new=[2, 3, 1, 4], kv=[100, 3, 1000, 257], heads=8, kv_heads=2, dim=128, page=128, order="hnd"),
    dict(new=[3, 16, 5], kv=[2, 16, 3], heads=1, kv_heads=1, dim=64, page=8),       # rows before the first position
    dict(new=[1, 2], kv=[5000, 3000], heads=8, kv_heads=1, dim=128, page=16, window=100),
    dict(new=[4], kv=[77], heads=2, kv_heads=2, dim=64, page=16, window=1),
    dict(new=[1, 4], kv=[300, 45], heads=4, kv_heads=2, dim=112, page=4096, causal=False),
    dict(new=[2], kv=[0], heads=4, kv_heads=2, dim=64, causal=False),
    dict(new=[1] * 3, kv=[40, 41, 42], heads=16, kv_heads=16, dim=104, page=8, pad=8),
    dict(new=[1, 1], kv=[3000, 2], heads=128, kv_heads=1, dim=128, page=256),       # more query heads than a tile
]


@pytest.mark.parametrize("c", FEW, ids=desc)
@pytest.mark.parametrize("waste", [0.0, NAN])
def test_attention_of_few_tokens(Q, c, waste):  # noqa: F811
    a = Attn(Q, seed=len(desc(c)), **c)
    a.spoil(waste)
    a.call()
    a.check()


@pytest.mark.parametrize("c", [
    dict(new=[1], kv=[200000], heads=8, kv_heads=8, dim=128, page=64),
    dict(new=[1] * 30, kv=[3000 + 17 * i for i in range(30)], heads=8, kv_heads=8, dim=128, page=16),
    dict(new=[1] * 30, kv=[6000 + 17 * i for i in range(30)], heads=12, kv_heads=6, dim=64, page=8, t="f16"),
], ids=desc)
def test_attention_of_single_tokens_over_many_tiles_a_block(Q, c):  # noqa: F811
    """rings that go round many times, with copies that land in any order"""
    a = Attn(Q, seed=8, **c)
    a.spoil(NAN)
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    a.call()
    a.check(only=range(min(a.batch, 3)))
    first = a.out.clone()
    for i in range(20):
        flush.fill_(i)
        a.out.zero_()
        a.call()
        assert torch.equal(a.out, first)
    for i in range(200):                                              # one behind the other
        a.call()
    assert torch.equal(a.out, first) and Q.moe_v41_read_status(a.ws) == 0


# chunks, prompts, drafts of several tokens
MANY = [
    dict(new=[128], kv=[128], heads=2, kv_heads=2, dim=128, page=16),
    dict(new=[100], kv=[300], heads=4, kv_heads=1, dim=64, page=32, t="f16", order="hnd"),
    dict(new=[257], kv=[1000], heads=3, kv_heads=1, dim=128, page=64),
    dict(new=[1000], kv=[1000], heads=4, kv_heads=4, dim=96, page=128, t="f16", order="hnd", padq=16),
    dict(new=[5] * 16, kv=[300 + 91 * i for i in range(16)], heads=32, kv_heads=4, dim=128, page=16),
    dict(new=[1, 700, 0, 33, 1], kv=[900, 700, 40, 2000, 1], heads=8, kv_heads=2, dim=128, page=16, tail=5),
    dict(new=[300], kv=[5000], heads=6, kv_heads=2, dim=80, page=8, window=129),
    dict(new=[400, 20], kv=[400, 3000], heads=2, kv_heads=1, dim=64, page=16, window=1000),
    dict(new=[64, 200], kv=[500, 33], heads=8, kv_heads=8, dim=64, page=8, order="hnd", causal=False),
    dict(new=[300], kv=[100], heads=2, kv_heads=1, dim=128, page=32),               # two thirds see nothing
    dict(new=[40], kv=[0], heads=2, kv_heads=1, dim=128, page=32),
    dict(new=[513], kv=[4000], heads=7, kv_heads=1, dim=40, page=16, t="f16"),
    dict(new=[2048], kv=[2048], heads=1, kv_heads=1, dim=128, page=512),
    dict(new=[17], kv=[17], heads=16, kv_heads=1, dim=16, page=8),
    dict(new=[130], kv=[131], heads=200, kv_heads=1, dim=32, page=8),
    dict(new=[50] * 20, kv=[50 + 13 * i for i in range(20)], heads=4, kv_heads=2, dim=72, page=16, t="f16"),
]


@pytest.mark.parametrize("c", MANY, ids=desc)
@pytest.mark.parametrize("waste", [0.0, NAN])
def test_attention_of_many_tokens(Q, c, waste):  # noqa: F811
    a = Attn(Q, seed=len(desc(c)), **c)
    a.spoil(waste)
    a.call()
    a.check()


@pytest.mark.parametrize("c", FEW + MANY, ids=desc)
def test_attention_with_another_idea_of_the_longest(Q, c):  # noqa: F811
    """max_new chooses a kernel, not a result"""
    for max_new in (1, 5000):
        a = Attn(Q, seed=len(desc(c)), max_new=max_new, **c)
        a.spoil(NAN)
        a.call()
        a.check()


# exact arithmetic: keys of zero make every weight one, so lse counts the keys that are seen
@pytest.mark.parametrize("max_new", [1, 5000])
@pytest.mark.parametrize("c", [
    dict(new=[70, 1, 300], kv=[1000, 4000, 300], heads=2, kv_heads=1, dim=64, page=8),
    dict(new=[70, 1, 300], kv=[1000, 4000, 300], heads=3, kv_heads=3, dim=128, page=16, window=77, t="f16"),
    dict(new=[200, 129], kv=[128, 5000], heads=5, kv_heads=1, dim=128, page=32, window=1),
    dict(new=[31, 129], kv=[127, 129], heads=1, kv_heads=1, dim=16, page=64, causal=False),
    dict(new=[600], kv=[20001], heads=1, kv_heads=1, dim=128, page=16),
], ids=desc)
def test_attention_counts_its_keys(Q, c, max_new):  # noqa: F811
    a = Attn(Q, max_new=max_new, **c)
    a.k.zero_()
    a.v.fill_(1.0)
    a.spoil(INF)
    a.call()
    for b in range(a.batch):
        at, n, ok = a.cu[b], a.new[b], a.visible(b)
        count = ok.sum(1).double()
        lse = a.lse[at:at + n].double()
        want = count.log()[:, None].expand_as(lse)
        # of 20000 keys one more or less is 5e-5
        assert (torch.where(count[:, None] > 0, lse - want, 0.0).abs() <= 4e-6).all()
        assert torch.equal(lse == -INF, (count == 0)[:, None].expand_as(lse))
        assert torch.equal(a.out[at:at + n].double(), (count > 0).double()[:, None].expand(n, a.out.shape[1]))


@pytest.mark.parametrize("max_new", [1, 5000])
def test_attention_follows_every_value_to_its_place(Q, max_new):  # noqa: F811
    """one key that outweighs the others by e^60 and more: its value comes out alone, for each head, token and position"""
    a = Attn(Q, [40], [900], 6, 2, 128, page=16, max_new=max_new, scale=1.0)
    pick = torch.randint(0, 861, (40, 6), generator=gen(9), device="cuda")      # seen by every token
    where = a.slots(0)
    bits = (torch.arange(900, device="cuda")[:, None] >> torch.arange(10, device="cuda")) & 1
    a.k.zero_()
    a.k[where[0], where[1], :, :10] = (bits * 2 - 1).to(a.k.dtype)[:, None].expand(900, 2, 10) * 8
    q = a.q.view(40, 6, 128)
    q.zero_()
    q[..., :10] = (((pick[..., None] >> torch.arange(10, device="cuda")) & 1) * 2 - 1).to(q.dtype) * 8
    a.call()
    got = a.out.view(40, 6, 128)
    for h in range(6):
        assert torch.equal(got[:, h], a.v[where[0], where[1], h // 3][pick[:, h]])


@pytest.mark.parametrize("max_new", [1, 5000])
@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_attention_of_rising_and_far_scores(Q, t, max_new):  # noqa: F811
    """scores that rise by hundreds along the keys, and differ by more than exp can hold"""
    a = Attn(Q, [3, 150], [2000, 700], 4, 2, 64, page=16, t=t, max_new=max_new, scale=1.0, spread=1.0)
    for b in range(2):
        where = a.slots(b)
        a.k[where[0], where[1], 0, 0] = torch.linspace(-300, 300, a.kv[b], device="cuda").to(T[t])
        a.k[where[0], where[1], 1, 0] = torch.linspace(300, -300, a.kv[b], device="cuda").to(T[t])
    a.q.view(a.m, 4, 64)[..., 0] = 1.0
    a.call()
    a.check()


@pytest.mark.parametrize("max_new", [1, 5000])
def test_attention_infinities_and_nans_stay_with_who_sees_them(Q, max_new):  # noqa: F811
    """a NaN in a query, and keys of another sequence and key head that hold infinities"""
    c = dict(new=[5, 200, 1], kv=[300, 200, 1000], heads=4, kv_heads=2, dim=128, page=16, max_new=max_new)
    a = Attn(Q, **c)
    a.call()
    clean, lse = a.out.clone().view(a.m, 4, 128), a.lse.clone()
    where = a.slots(1)
    a.k[where[0][3], where[1][3], 1] = INF
    a.v[where[0][7], where[1][7], 0] = NAN
    a.q.view(a.m, 4, 128)[2, 1] = NAN
    a.call()
    got = a.out.view(a.m, 4, 128)
    assert torch.isnan(got[2, 1]).all() and torch.isnan(a.lse[2, 1])
    fine = torch.ones((a.m, 4), dtype=torch.bool, device="cuda")
    fine[2, 1] = False
    fine[5:205] = False
    assert torch.equal(got[fine], clean[fine]) and torch.equal(a.lse[fine], lse[fine])
    assert torch.isnan(got[5 + 7:205, :2]).all()                      # who sees the NaN value
    assert torch.equal(a.lse[5:205, :2], lse[5:205, :2])              # scores know nothing of values
    assert not torch.isfinite(a.lse[5 + 3:205, 2:]).any()


@pytest.mark.parametrize("c,max_new", [
    (dict(new=[1], kv=[50000], heads=8, kv_heads=1, dim=128, page=16), 1),
    (dict(new=[1, 2, 1], kv=[3000, 700, 9], heads=8, kv_heads=2, dim=64, page=16), 2),
    (dict(new=[500], kv=[9000], heads=4, kv_heads=1, dim=128, page=32), 500)], ids=str)
def test_attention_repeats_bit_for_bit(Q, c, max_new):  # noqa: F811
    """on one workspace, call after call, whichever block is the last"""
    a = Attn(Q, max_new=max_new, **c)
    a.call()
    a.check()
    first = a.out.clone(), a.lse.clone()
    for _ in range(30):
        a.out.zero_()
        a.lse.zero_()
        a.call()
        assert torch.equal(a.out, first[0]) and torch.equal(a.lse, first[1])


def test_attention_without_lse_and_without_tokens(Q):  # noqa: F811
    a = Attn(Q, [3, 1], [50, 60], 4, 2, 64)
    a.call(lse=False)
    assert (a.lse == 77.0).all()
    a.call()
    a.check()
    none = Attn(Q, [0, 0], [50, 0], 4, 2, 64, tail=4)
    none.call()
    torch.cuda.synchronize()
    assert (none.out == 77.0).all() and Q.moe_v41_read_status(none.ws) == 0


@pytest.mark.parametrize("max_new", [1, 5000])
def test_attention_of_bad_pages(Q, max_new):  # noqa: F811
    """pages that are none read as zeros, and the status says so; the other sequences are right"""
    a = Attn(Q, [1, 40, 1], [100, 100, 100], 4, 2, 64, page=16, max_new=max_new)
    clean = a.table.clone()
    a.call()
    want = a.out.clone()
    a.table[1, 2] = -1
    a.table[1, 4] = a.n_pages
    a.table[1, 5] = 2 ** 31 - 1
    a.call()
    assert torch.equal(a.out[0], want[0]) and torch.equal(a.out[41], want[41])
    assert Q.moe_v41_read_status(a.ws, clear=True) == Q.MOE_STATUS_BAD_PAGE
    got = a.out.clone()
    a.table.copy_(clean)
    for i in (2, 4, 5):
        a.k[a.table[1, i]] = 0
        a.v[a.table[1, i]] = 0
    a.call()
    a.check()
    assert torch.equal(a.out[1:41], got[1:41])


@pytest.mark.parametrize("max_new", [1, 5000])
def test_attention_of_a_length_beyond_the_table(Q, max_new):  # noqa: F811
    """what has no entry in the table is not seen, and the status says so"""
    a = Attn(Q, [3, 40], [100, 64], 4, 2, 64, page=16, max_new=max_new)
    more = 16 * a.cols + 30
    a.ints[1][0] = more
    a.call()
    assert Q.moe_v41_read_status(a.ws, clear=True) == Q.MOE_STATUS_BAD_PAGE
    a.kv[0] = 16 * a.cols                                             # the three tokens lie behind these, and see all of them
    ok = torch.ones((3, a.kv[0]), dtype=torch.bool, device="cuda")
    visible = a.visible
    a.visible = lambda b: ok if b == 0 else visible(b)
    a.check()


# ------------------------------------------------------------------ append

APPEND = [
    dict(new=[1], kv=[1], heads=4, kv_heads=1, dim=64, page=8),
    dict(new=[1] * 48, kv=list(range(1, 49)), heads=32, kv_heads=8, dim=128, page=16),
    dict(new=[1] * 1100, kv=[i % 70 + 1 for i in range(1100)], heads=2, kv_heads=2, dim=16, page=16),
    dict(new=[300, 0, 1, 77], kv=[300, 5, 900, 400], heads=6, kv_heads=3, dim=80, page=64, t="f16", order="hnd", tail=4),
    dict(new=[33, 0, 0, 5], kv=[33, 0, 1, 6], heads=3, kv_heads=1, dim=24, page=32, tail=1),
    dict(new=[20, 4], kv=[7, 40], heads=1, kv_heads=1, dim=128, page=4096),        # tokens before the first position
]


@pytest.mark.parametrize("c", APPEND, ids=desc)
@pytest.mark.parametrize("x,rot,first,layout", [("f32", None, 0, 0), ("bf16", None, 0, 1), ("f16", 8, 8, 0), ("f32", 6, 2, 1),
                                                ("bf16", 0, 0, 0)])
def test_append_against_64_bits(Q, c, x, rot, first, layout):  # noqa: F811
    a = Cache(Q, seed=3, **c)
    t = T[a.t]
    rot = a.dim if rot is None else rot
    f, mag = Q.moe_v41_rope_freqs(rot, 10000.0, Q.MOE_ROPE_SCALE_PARTS, 4.0, 64)
    f = torch.tensor(f, dtype=torch.float64, device="cuda")
    qkv = torch.randn((a.m, a.heads + 2 * a.kv_heads, a.dim), generator=a.g, device="cuda").to(T[x])
    qkv[a.cu[-1]:] = NAN
    q, k, v = qkv[:, :a.heads], qkv[:, a.heads:a.heads + a.kv_heads], qkv[:, a.heads + a.kv_heads:]
    q_out = torch.full((a.m, a.heads, a.dim), 77.0, dtype=t, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = [c_.clone() for c_ in a.caches]
    cfg = Q.make_rope_cfg(a.dim, rot, first, layout, code(Q, x), magnitude=mag)

    def call(q_=q, q_out_=q_out, pos=None):
        Q.moe_v41_kv_append(a.kv_cfg, cfg, a.seqs, a.m, k, k.stride(0), v, v.stride(0), a.k, a.v, a.heads, q_, q.stride(0),
                            q_out_, a.heads * a.dim, f, pos, status)

    call()
    n = a.cu[-1]
    pos = a.positions()
    tols = [None, None]
    for b in range(a.batch):
        at, first_pos = a.cu[b], a.kv[b] - a.new[b]
        skip = max(0, -first_pos)
        if a.new[b] - skip <= 0:
            continue
        rows, p = slice(at + skip, at + a.new[b]), torch.arange(first_pos + skip, a.kv[b], device="cuda")
        page, slot = a.table[b].long()[p // a.page], p % a.page
        wk = turned(k[rows], p, f, first, layout, mag)
        tol = rope_tol(k[rows], p, f, first, layout, mag, a.t) + half_step(a.t, wk) * 1.001
        close(a.k[page, slot].double(), wk, tol, f"keys of sequence {b}")
        assert torch.equal(a.v[page, slot], v[rows].to(t))
        want[0][page, slot], want[1][page, slot] = a.k[page, slot], v[rows].to(t)
    del tols
    assert torch.equal(a.k, want[0]) and torch.equal(a.v, want[1])                # and nothing else was written
    wq = turned(q[:n], pos, f, first, layout, mag)
    close(q_out[:n].double(), wq, rope_tol(q[:n], pos, f, first, layout, mag, a.t) + half_step(a.t, wq) * 1.001, "q")
    assert (q_out[n:] == 77.0).all() and int(status) == 0
    # keys alone; positions of their own
    q_out.fill_(77.0)
    for c_ in a.caches:
        c_.zero_()
    shift = torch.zeros(a.m, dtype=torch.int32, device="cuda")
    shift[:n] = pos + 1000
    call(None, None, shift)
    assert (q_out == 77.0).all()
    b = max(range(a.batch), key=lambda i: a.kv[i] if a.new[i] else -1)
    p = torch.arange(max(0, a.kv[b] - a.new[b]), a.kv[b], device="cuda")
    rows = slice(a.cu[b + 1] - p.numel(), a.cu[b + 1])
    page, slot = a.table[b].long()[p // a.page], p % a.page
    wk = turned(k[rows], p + 1000, f, first, layout, mag)
    close(a.k[page, slot].double(), wk, rope_tol(k[rows], p + 1000, f, first, layout, mag, a.t)
          + half_step(a.t, wk) * 1.001, "keys at positions of their own")


def test_append_rotates_queries_in_place(Q):  # noqa: F811
    a = Cache(Q, [3, 9], [30, 9], 4, 2, 64)
    f, _ = Q.moe_v41_rope_freqs(64)
    f = torch.tensor(f, dtype=torch.float64, device="cuda")
    qkv = torch.randn((a.m, 8, 64), generator=gen(2), device="cuda").bfloat16()
    before = qkv.clone()
    Q.moe_v41_kv_append(a.kv_cfg, Q.make_rope_cfg(64), a.seqs, a.m, qkv[:, 4:], 512, qkv[:, 6:], 512, a.k, a.v, 4, qkv, 512,
                        qkv, 512, f, None, None)
    want = turned(before[:, :4], a.positions(), f, 0, 0)
    close(qkv[:, :4].double(), want, rope_tol(before[:, :4], a.positions(), f, 0, 0, 1.0, "bf16")
          + half_step("bf16", want) * 1.001, "q")
    assert torch.equal(qkv[:, 4:], before[:, 4:])


def test_append_of_bad_pages(Q):  # noqa: F811
    """what has no page is not stored, the status says so, and the rest is"""
    a = Cache(Q, [3, 20, 2], [3, 20, 40], 2, 2, 64, page=8, extra_pages=5)
    clean = [c.clone() for c in a.caches]
    k = torch.randn((a.m, 2, 64), generator=gen(2), device="cuda").bfloat16()
    cfg, status = Q.make_rope_cfg(64, 0), torch.zeros(1, dtype=torch.int32, device="cuda")
    a.table[1, 0] = -3
    a.table[1, 2] = a.n_pages
    a.ints[1][2] = a.cols * 8 + 1                                                 # the last token is beyond the table
    last = a.slots(2, a.cols * 8)
    Q.moe_v41_kv_append(a.kv_cfg, cfg, a.seqs, a.m, k, 128, k, 128, a.k, a.v, 0, None, 0, None, 0, None, None, status)
    assert int(status) == Q.MOE_STATUS_BAD_PAGE
    for c, old in zip(a.caches, clean):
        old[a.table[0].long()[0], :3] = k[:3]
        old[a.table[1].long()[1]] = k[3 + 8:3 + 16]
        if int(a.table[2, a.cols - 1]) >= 0:
            old[last[0][-1], last[1][-1]] = k[23]
        assert torch.equal(c, old)


# ------------------------------------------------------------------ beyond 32 bits, other streams

@pytest.mark.parametrize("max_new", [1, 5000])
def test_attention_far_into_a_large_cache(Q, max_new):  # noqa: F811
    """pages whose values lie beyond 2^32 bytes and 2^31 values"""
    pages, page, kv_heads, dim = 70000, 64, 4, 128                                # 4.6 GB each for keys and values
    a = Attn(Q, [1, 70], [1000, 3000], 8, kv_heads, dim, page=page, max_new=max_new)
    big = [torch.zeros((pages, page, kv_heads, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    move = torch.arange(a.n_pages, device="cuda") * 7 + (pages - 7 * a.n_pages)   # the last pages
    for small, large in zip(a.caches, big):
        large[move] = small
    a.table.copy_(torch.where(a.table >= 0, move[a.table.clamp(min=0).long()].int(), a.table))
    a.caches = a.k, a.v = big
    a.n_pages = pages
    a.kv_cfg = Q.make_kv_cfg(kv_heads, dim, page, pages)
    a.cfg = Q.make_attn_cfg(a.kv_cfg, 8, True, 0, a.scale)
    a.call()
    a.check()
    k = torch.randn((a.m, kv_heads, dim), generator=gen(1), device="cuda").bfloat16()
    Q.moe_v41_kv_append(a.kv_cfg, Q.make_rope_cfg(dim, 0), a.seqs, a.m, k, kv_heads * dim, k, kv_heads * dim, a.k, a.v, 0,
                        None, 0, None, 0, None, None, None)
    p, s = a.slots(1)
    assert torch.equal(a.k[p[-70:], s[-70:]], k[1:]) and torch.equal(a.v[p[-70:], s[-70:]], k[1:])


def test_a_captured_step_serves_growing_sequences(Q):  # noqa: F811
    """append and attention in one graph, replayed as the lengths grow on the device, on a stream of its own"""
    heads, kv_heads, dim, page, steps = 8, 2, 64, 16, 40
    a = Attn(Q, [1, 1, 1], [60, 41, 1 + steps], heads, kv_heads, dim, page=page)
    f, _ = Q.moe_v41_rope_freqs(dim)
    f = torch.tensor(f, dtype=torch.float64, device="cuda")
    qkv = torch.zeros((3, heads + 2 * kv_heads, dim), dtype=torch.bfloat16, device="cuda")
    start = torch.tensor([60 - steps, 41 - steps, 1], dtype=torch.int32, device="cuda")
    a.ints[1].copy_(start)
    row = qkv.stride(0)
    cfg = Q.make_rope_cfg(dim)
    kv_ptr = [qkv[:, heads:], qkv[:, heads + kv_heads:]]
    q = torch.empty((3, heads * dim), dtype=torch.bfloat16, device="cuda")

    def step():
        Q.moe_v41_kv_append(a.kv_cfg, cfg, a.seqs, 3, kv_ptr[0], row, kv_ptr[1], row, a.k, a.v, heads, qkv, row, q,
                            heads * dim, f, None, None)
        Q.moe_v41_paged_attention(a.cfg, a.seqs, 3, 1, q, heads * dim, a.k, a.v, a.out, heads * dim, a.lse, heads, a.ws)

    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        step()
    given = torch.randn((steps, 3, heads + 2 * kv_heads, dim), generator=gen(6), device="cuda").bfloat16()
    for i in range(steps):
        qkv.copy_(given[i])
        graph.replay()
        a.ints[1] += 1
    torch.cuda.synchronize()
    a.q = q
    a.ints[1] -= 1
    a.kv = a.ints[1].tolist()
    assert a.kv == [60 - 1, 41 - 1, steps]
    a.check()
    # the whole history of the third sequence, from what was given
    p, s = a.slots(2)
    want = turned(given[:, 2, heads:heads + kv_heads], torch.arange(steps, device="cuda"), f, 0, 0)
    assert ((a.k[p, s].double() - want).abs() <= 2.0 ** -8 * 1.01 * want.abs() + 1e-5).all()
    assert torch.equal(a.v[p, s], given[:, 2, heads + kv_heads:])

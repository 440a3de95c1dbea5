"""The operators around the MoE layer on the GPU against plain 64-bit torch.

Tolerances are derived from the rounding of 32-bit sums: u = 2^-24 is half a
step of f32 relative to a value, and an output of a narrower type adds half a
step of that type (2^-8 bf16, 2^-11 fp16; fp16 has no relative step below
2^-14, where its half step is 2^-25).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = 2.0 ** -24
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def Q():
    import quantized_mixture_experts_router_gb300 as Q
    Q.lib()
    return Q


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def code(Q, t):
    return {"f32": Q.MOE_T_F32, "bf16": Q.MOE_T_BF16, "f16": Q.MOE_T_F16}[t]


def half_step(t, value):
    """half a step of type t at each value"""
    if t == "f32":
        return U * value.abs()
    if t == "bf16":
        return 2.0 ** -8 * value.abs()
    return torch.clamp(2.0 ** -11 * value.abs(), min=2.0 ** -25)


def close(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at "
                           f"{bad.nonzero()[0].tolist()}: got {got[bad][0].item()!r}, want {want[bad][0].item()!r}, "
                           f"tolerance {tol[bad][0].item() if torch.is_tensor(tol) else tol!r}")


def pitched(rows, cols, pitch, dtype, fill):
    full = torch.full((rows, pitch), fill, dtype=dtype, device="cuda")
    return full, full[:, :cols]


# ------------------------------------------------------------------ 4-bit linear

class Q4:
    def __init__(self, Q, m, n, k, group, zeros=False, x="bf16", s="f16", out="f32", padx=0, pado=0, seed=0,
                 max_tokens=None):
        g = gen(seed)
        self.Q, self.m, self.n, self.k, self.group, self.xt, self.st, self.ot = Q, m, n, k, group, x, s, out
        self.ng = -(-k // group)
        _, self.x = pitched(m, k, k + padx, T[x], NAN)
        self.x.copy_(torch.randn((m, k), generator=g, device="cuda"))
        self.w = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
        self.scales = (torch.rand((n, self.ng), generator=g, device="cuda") * 0.02 + 0.005).to(T[s])
        self.zeros = torch.randint(0, 16, (n, self.ng), generator=g, device="cuda",
                                   dtype=torch.uint8) if zeros else None
        self.full, self.out = pitched(m, n, n + pado, T[out], 77.0)
        self.cfg = Q.make_q4_cfg(n, k, group, code(Q, x), code(Q, s), code(Q, out), max_tokens=max_tokens or max(m, 1))
        self.ws = torch.empty(Q.moe_v41_q4_workspace_bytes(self.cfg), dtype=torch.uint8, device="cuda")
        Q.moe_v41_workspace_init(self.ws)

    def call(self, m=None, stream=None):
        self.Q.moe_v41_q4_linear(self.cfg, self.x, self.m if m is None else m, self.x.stride(0), self.w, self.scales,
                                 self.zeros, self.out, self.out.stride(0), self.ws, stream=stream)

    def weights(self):
        q = torch.stack((self.w & 15, self.w >> 4), -1).reshape(self.n, self.k).double()
        z = (self.zeros.double() if self.zeros is not None else torch.full_like(self.scales, 8.0).double())
        idx = torch.arange(self.k, device="cuda") // self.group
        return (q - z[:, idx]) * self.scales.double()[:, idx]

    def check(self):
        w, x = self.weights(), self.x.double()
        want, mag = x @ w.t(), x.abs() @ w.abs().t()
        # k products in any order of f32 sums that round or cut (2 u each), the group factor and the joins: the
        # rigorous bound; in norm the roundings of random terms add up far less: k / 16 cut sums of partial results
        # below the final one, 2 u each, at most 2048 of them here
        tol = 2 * U * (self.k + 64) * mag + half_step(self.ot, want)
        close(self.out, want, tol, "q4")
        rel = (self.out.double() - want).norm() / want.norm()
        assert rel <= 2 * U * max(32, self.k / 16) + {"f32": U, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[self.ot]
        if self.full.shape[1] > self.n:
            assert (self.full[:, self.n:] == 77.0).all()
        assert self.Q.moe_v41_read_status(self.ws) == 0


Q4_CASES = [
    # m, n, k, group, zeros, x, s, out, padx, pado
    (1, 1, 32, 32, False, "bf16", "f16", "f32", 0, 0),
    (1, 7, 32, 128, True, "f16", "bf16", "f16", 0, 0),
    (1, 33, 64, 64, True, "bf16", "bf16", "bf16", 8, 3),
    (1, 512, 5120, 128, False, "bf16", "f16", "f32", 0, 0),
    (1, 2305, 2304, 64, True, "f16", "f16", "f32", 0, 1),
    (1, 64, 32768, 32, True, "bf16", "f16", "f32", 0, 0),
    (1, 20001, 512, 128, True, "bf16", "f16", "f32", 0, 0),
    (2, 31, 96, 64, True, "bf16", "f16", "f32", 0, 0),
    (3, 100, 160, 128, True, "f16", "f16", "f32", 24, 5),
    (4, 512, 512, 32, False, "bf16", "f16", "bf16", 0, 0),
    (5, 5001, 2336, 128, True, "bf16", "f16", "f32", 24, 24),
    (7, 160, 1056, 32, False, "bf16", "bf16", "f16", 0, 0),
    (8, 4608, 5120, 32, True, "f16", "f16", "f32", 0, 0),
    (8, 16, 32768, 128, False, "bf16", "f16", "f32", 0, 0),
    (8, 9999, 7680, 64, True, "bf16", "f16", "f32", 0, 0),
    (9, 129, 256, 128, True, "bf16", "f16", "f32", 0, 1),
    (16, 1000, 2048, 64, False, "bf16", "f16", "f32", 0, 0),
    (17, 300, 480, 32, True, "f16", "bf16", "f32", 8, 7),
    (33, 129, 32, 32, False, "bf16", "f16", "f16", 0, 0),
    (64, 640, 5120, 128, True, "bf16", "f16", "bf16", 0, 0),
    (100, 127, 1312, 128, True, "f16", "f16", "f16", 8, 1),
    (128, 256, 1024, 64, True, "bf16", "bf16", "f32", 0, 0),
    (257, 1153, 608, 128, True, "bf16", "f16", "f32", 0, 0),
    (300, 2304, 2304, 32, True, "bf16", "f16", "f32", 16, 8),
    (512, 5120, 5120, 128, False, "bf16", "f16", "f32", 0, 0),
    (1000, 40, 128, 64, True, "bf16", "f16", "f32", 0, 0),
]


@pytest.mark.parametrize("c", Q4_CASES, ids=str)
def test_q4_against_64_bits(Q, c):
    t = Q4(Q, *c, seed=sum(c[:4]))
    t.call()
    t.check()


def test_q4_every_code_and_zero(Q):
    """all 256 code pairs against all 16 zeros: each product is exact, one term per sum"""
    n, k = 256, 512
    t = Q4(Q, 1, n, k, 32, zeros=True)
    t.w[:] = torch.arange(256, device="cuda", dtype=torch.uint8)[:, None]
    t.scales.fill_(0.5)
    t.zeros[:] = torch.arange(16, device="cuda", dtype=torch.uint8)[None, :]
    for j in range(k // 32):
        for odd in (0, 1):
            t.x.zero_()
            t.x[0, 32 * j + 2 * (j % 16) + odd] = 2.0
            t.call()
            q = torch.arange(256, device="cuda") >> (4 * odd) & 15
            assert torch.equal(t.out[0], (q - j).float())


@pytest.mark.parametrize("m", [2, 8, 40])
def test_q4_nan_and_inf_stay_in_their_row(Q, m):
    t = Q4(Q, m, 200, 320, 64, zeros=True, seed=5)
    t.call()
    clean = t.out.clone()
    t.x[1, 17] = NAN
    t.x[0, 3] = INF
    t.scales[9, 2] = INF
    t.call()
    w, x = t.weights(), t.x.double()
    want = torch.stack([(x[i] * w).sum(1) for i in range(2)])
    assert torch.isnan(t.out[1]).all()
    keep = [r for r in range(200) if r != 9]
    assert torch.equal(torch.isnan(want[0, keep]), torch.isnan(t.out[0, keep]))
    fine = ~torch.isnan(want[0])
    fine[9] = False
    assert torch.equal(want[0, fine].float(), t.out[0, fine])      # +-inf
    assert torch.equal(t.out[2:, keep], clean[2:, keep])
    assert not torch.isfinite(t.out[:, 9]).any()


@pytest.mark.parametrize("shape", [(1, 64, 32768, 128), (8, 5000, 2304, 32), (3, 20001, 544, 64),
                                   (200, 700, 1024, 128)], ids=str)
def test_q4_repeats_bit_for_bit_and_shares_a_workspace(Q, shape):
    t = Q4(Q, *shape, zeros=True, seed=3)
    t.call()
    t.check()
    first = t.out.clone()
    for _ in range(20):
        t.out.zero_()
        t.call()
        assert torch.equal(t.out, first)
    for m in sorted({1, max(1, t.m // 2), t.m}):                   # fewer tokens on the same workspace
        t.out.fill_(7.0)
        t.call(m=m)
        assert (t.out[m:] == 7.0).all()
        want = t.x[:m].double() @ t.weights().t()
        assert ((t.out[:m].double() - want).norm() / want.norm()) <= 2 * U * max(32, t.k / 16)


def test_q4_of_no_tokens_writes_nothing(Q):
    t = Q4(Q, 2, 64, 64, 32)
    t.call(m=0)
    torch.cuda.synchronize()
    assert (t.out == 77.0).all()


@pytest.mark.parametrize("shape", [(1, 512, 5120, 128), (6, 3000, 1024, 32), (70, 300, 512, 64)], ids=str)
def test_q4_on_another_stream_and_in_a_graph(Q, shape):
    t = Q4(Q, *shape, seed=11)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    t.call(stream=s)
    s.synchronize()
    want = t.out.clone()
    t.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        t.call(stream=s)
    t.out.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(t.out, want)
    t.x.mul_(2.0)                                                  # new inputs in the same buffers
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(t.out, want * 2.0)


# ------------------------------------------------------------------ block norm

def n64(v, kind, w, b, eps):
    if kind == 0:
        return v
    if kind == 2:
        v = v - v.mean(1, keepdim=True)
    v = v / ((v * v).mean(1, keepdim=True) + eps).sqrt()
    if w is not None:
        v = v * w.double()
    return v if b is None else v + b.double()


def n64_tol(v, kind, w, b, eps, tv):
    """how far f32 may be from n64(v) when v itself is off by tv: the sums of dim positive terms in at most 64 steps
    (per thread, warp and block) and eight roundings of the factor, 72 u <= 2^-17, of the centred value and of the
    mean taken off it; and tv passed on through the value (1), the mean (1) and the scale (1)"""
    if kind == 0:
        return tv
    mean = v.mean(1, keepdim=True) if kind == 2 else torch.zeros_like(v[:, :1])
    c = v - mean
    r = 1.0 / ((c * c).mean(1, keepdim=True) + eps).sqrt()
    aw = w.double().abs() if w is not None else 1.0
    t = 2.0 ** -17 * r * (c.abs() + v.abs().mean(1, keepdim=True) * (kind == 2)) * aw
    big = tv.max(1, keepdim=True).values
    t = t + aw * r * (2 * tv + big + c.abs() * r * big) * 1.01
    return t if b is None else t + U * 2 * (b.double().abs() + (c * r).abs() * aw)


class Norm:
    def __init__(self, Q, m, dim, post="rms", pre="rms", y="f32", h="bf16", x="bf16", w="f32", gate="none", gt="f32",
                 group=1, bias=False, pad=0, seed=0, eps=1e-6, offset=0.0, alpha=0.75, beta=1.25, off=0):
        K = {"none": Q.MOE_NORM_NONE, "rms": Q.MOE_NORM_RMS, "layer": Q.MOE_NORM_LAYER}
        g = gen(seed)
        self.Q, self.m, self.dim, self.eps, self.alpha, self.beta = Q, m, dim, eps, alpha, beta
        self.yt, self.ht, self.xt, self.gate_kind, self.group = y, h, x, gate, group

        def mat(rows, t, spread, mean):
            buf = torch.full((rows * (dim + pad) + off,), 55.0, dtype=T[t], device="cuda")[off:]
            v = buf.view(rows, dim + pad)[:, :dim]
            v.copy_(torch.randn((rows, dim), generator=g, device="cuda") * spread + mean)
            return v

        def vec(t, mean):
            return (torch.randn((dim,), generator=g, device="cuda") * 0.3 + mean).to(T[t])

        self.y, self.h = mat(m, y, 0.5, offset), mat(m, h, 2.0, -offset)
        self.post_w, self.pre_w = vec(w, 1.0), vec(w, 1.0)
        self.post_b, self.pre_b = (vec(w, 0.1), vec(w, -0.1)) if bias else (None, None)
        self.gate = None
        if gate == "row":
            self.gate = mat(-(-m // group), gt, 0.2, 0.6)
        elif gate == "token":
            self.gate = (torch.rand((-(-m // group),), generator=g, device="cuda") + 0.3).to(T[gt])
        self.h_out, self.x_out = mat(m, h, 0.0, 55.0), mat(m, x, 0.0, 55.0)
        self.post, self.pre = K[post], K[pre]
        self.cfg = Q.make_norm_cfg(dim, self.post, self.pre, code(Q, y), code(Q, h), code(Q, x), code(Q, w),
                                   {"none": 0, "row": 1, "token": 2}[gate], code(Q, gt), group, eps, alpha, beta)

    def call(self, stream=None, **kw):
        a = dict(y=self.y, h_out=self.h_out, x_out=self.x_out, post_w=self.post_w, pre_w=self.pre_w)
        a.update(kw)

        def ld(t):
            return 0 if t is None else t.stride(0)

        self.Q.moe_v41_block_norm(self.cfg, self.m, a["y"], ld(a["y"]), a["post_w"], self.post_b, self.gate,
                                  ld(self.gate), self.h, ld(self.h), a["h_out"], ld(a["h_out"]), a["pre_w"],
                                  self.pre_b, a["x_out"], ld(a["x_out"]), stream=stream)

    def want(self, y=True, post_w=True, pre_w=True):
        h = self.h.double()
        pw, qw = self.post_w if post_w else None, self.pre_w if pre_w else None
        a = float(torch.tensor(self.alpha, dtype=torch.float32))
        b = float(torch.tensor(self.beta, dtype=torch.float32))
        if not y:
            hn = a * h
            th = U * 2 * hn.abs()
        else:
            v = self.y.double()
            ny = n64(v, self.post, pw, self.post_b, self.eps)
            ty = n64_tol(v, self.post, pw, self.post_b, self.eps, torch.zeros_like(v))
            gt = 1.0
            if self.gate is not None:
                rows = torch.arange(self.m, device="cuda") // self.group
                gt = self.gate.double()[rows]
                gt = gt if gt.dim() == 2 else gt[:, None]
            hn = a * h + b * gt * ny
            th = (b * gt * ty).abs() if torch.is_tensor(gt) else b * ty
            th = th + 4 * U * ((a * h).abs() + (b * gt * ny).abs())
        x = n64(hn, self.pre, qw, self.pre_b, self.eps)
        tx = n64_tol(hn, self.pre, qw, self.pre_b, self.eps, th)
        return hn, th + half_step(self.ht, hn), x, tx + half_step(self.xt, x)

    def check(self, **kw):
        hn, th, x, tx = self.want(**kw)
        close(self.h_out, hn, th * 1.001, "h")
        close(self.x_out, x, tx * 1.001, "x")


NORM_CASES = [
    dict(m=1, dim=1), dict(m=3, dim=7, post="layer", pre="layer", bias=True), dict(m=2, dim=8, gate="row"),
    dict(m=5, dim=255, gate="token", y="bf16"), dict(m=1, dim=256, post="layer", bias=True, gate="row", group=4),
    dict(m=1, dim=5120, gate="row", group=1), dict(m=1, dim=5120, y="f32", h="f32", x="f16"),
    dict(m=9, dim=2305, post="layer", pre="layer", y="bf16", h="bf16", x="f16", w="bf16", gate="row", group=4, bias=True),
    dict(m=300, dim=5120, y="f32", h="f32", gate="token", gt="bf16", group=7),
    dict(m=700, dim=2304, y="bf16", h="bf16", w="bf16", gate="row", gt="f16", group=64),
    dict(m=1000, dim=512, y="f32", h="f32", post="none", gate="row", group=2000),
    dict(m=1200, dim=1000, y="f16", h="f32", x="f32", bias=True),
    dict(m=401, dim=7680, y="f32", h="bf16", post="rms", pre="layer", bias=True),
    dict(m=310, dim=4096, y="f32", h="f32", pre="none", x="f32"),
    dict(m=2, dim=8200, y="f16", h="f16", x="f16", w="f16"), dict(m=3, dim=16384, y="f32", h="f32", x="f32"),
    dict(m=320, dim=16384, y="bf16"), dict(m=2, dim=16383, y="bf16", post="layer", bias=True),
    dict(m=33, dim=512, pad=8, gate="row"), dict(m=333, dim=512, pad=8, gate="token"),
    dict(m=400, dim=640, pad=4, y="bf16", h="bf16"),
    dict(m=33, dim=512, pad=1), dict(m=33, dim=512, off=1, y="bf16"), dict(m=320, dim=1024, off=3, y="f32", h="f32"),
    dict(m=4, dim=3001, pre="none", post="none", gate="token"), dict(m=4, dim=512, pre="rms", post="none", x="f32"),
    # a common offset a thousand times the spread
    dict(m=4, dim=1024, post="layer", pre="layer", h="f32", offset=500.0),
    dict(m=301, dim=1024, post="layer", pre="layer", h="f32", offset=500.0),
]


@pytest.mark.parametrize("c", NORM_CASES, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_norm_against_64_bits(Q, c):
    t = Norm(Q, seed=c["m"] + c["dim"], **c)
    t.call()
    t.check()


@pytest.mark.parametrize("m,dim", [(1, 512), (500, 512), (3, 333), (500, 8192)])
def test_norm_parts_may_be_left_out(Q, m, dim):
    t = Norm(Q, m, dim, gate="token", bias=True, seed=1)
    t.call(y=None)                                                 # the first block's input: no output to add
    t.check(y=False)
    t.call(post_w=None, pre_w=None)
    t.check(post_w=False, pre_w=False)
    hn, th, x, tx = t.want()
    t.h_out.fill_(9.0)
    t.x_out.fill_(9.0)
    t.call(x_out=None)                                             # the last block: no norm follows
    close(t.h_out, hn, th * 1.001, "h")
    assert (t.x_out == 9.0).all()
    t.h_out.fill_(9.0)
    t.call(h_out=None)
    close(t.x_out, x, tx * 1.001, "x")
    assert (t.h_out == 9.0).all()


@pytest.mark.parametrize("m,dim", [(1, 5120), (700, 5120), (40, 777)])
def test_norm_in_place_and_pads_untouched(Q, m, dim):
    t = Norm(Q, m, dim, pad=8, gate="row", group=3, seed=2)
    t.call()
    want = t.h_out.clone(), t.x_out.clone()
    base = t.h._base if t.h._base is not None else t.h
    t.call(h_out=t.h)
    assert torch.equal(t.h, want[0]) and torch.equal(t.x_out, want[1])
    assert (base.view(-1).reshape(m, dim + 8)[:, dim:] == 55.0).all()


@pytest.mark.parametrize("m", [4, 600])
def test_norm_zero_nan_and_huge_rows(Q, m):
    t = Norm(Q, m, 1024, y="f32", h="f32", x="f32", gate="token", seed=4)
    t.y[0] = 0.0
    t.y[1, 5] = NAN
    t.y[2] *= 1e15
    t.call()
    assert torch.isnan(t.h_out[1]).all() and torch.isnan(t.x_out[1]).all()
    hn, th, x, tx = t.want()
    rest = [i for i in range(m) if i != 1]
    close(t.h_out[rest], hn[rest], th[rest] * 1.001, "h")
    close(t.x_out[rest], x[rest], tx[rest] * 1.001, "x")


def test_norm_on_another_stream_and_in_a_graph(Q):
    for m in (1, 512):
        t = Norm(Q, m, 5120, gate="row", group=m, seed=6)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        t.call(stream=s)
        s.synchronize()
        t.check()
        want = t.h_out.clone(), t.x_out.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            t.call(stream=s)
        t.h_out.zero_()
        t.x_out.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(t.h_out, want[0]) and torch.equal(t.x_out, want[1])


# ------------------------------------------------------------------ token log probabilities

class Lp:
    def __init__(self, Q, m, v, t="f32", k=5, temp=1.0, mask=False, pad=0, off=0, seed=0, spread=3.0, logits=None):
        g = gen(seed)
        self.Q, self.m, self.v, self.t, self.k = Q, m, v, t, k
        self.temp = float(torch.tensor(temp, dtype=torch.float32))
        buf = torch.full((m * (v + pad) + off,), NAN, dtype=T[t], device="cuda")[off:]
        self.x = buf.view(m, v + pad)[:, :v]
        self.x.copy_(torch.randn((m, v), generator=g, device="cuda") * spread if logits is None else logits)
        self.target = torch.randint(0, v, (m,), generator=g, device="cuda", dtype=torch.int32)
        self.bits = None
        if mask:
            w = torch.randint(-(1 << 31), 1 << 31, (m, -(-v // 32) + 1), generator=g, device="cuda")
            self.bits = w.to(torch.int32)
        f = dict(dtype=torch.float32, device="cuda")
        i = dict(dtype=torch.int32, device="cuda")
        self.logprob, self.lse, self.entropy = (torch.full((m,), 5.0, **f) for _ in range(3))
        self.rank = torch.full((m,), 5, **i)
        self.top, self.ids = torch.full((m, k), 5.0, **f), torch.full((m, k), 5, **i)
        self.cfg = Q.make_logprob_cfg(v, code(Q, t), k, temp)

    def call(self, stream=None, **kw):
        a = dict(target=self.target, logprob=self.logprob, rank=self.rank, lse=self.lse, entropy=self.entropy)
        a.update(kw)
        self.Q.moe_v41_token_logprobs(self.cfg, self.x, self.m, self.x.stride(0), self.bits,
                                      0 if self.bits is None else self.bits.stride(0), a["target"], a["logprob"],
                                      a["rank"], a["lse"], a["entropy"], self.top, self.ids, stream=stream)

    def allowed(self):
        if self.bits is None:
            return torch.ones((self.m, self.v), dtype=torch.bool, device="cuda")
        j = torch.arange(self.v, device="cuda")
        return ((self.bits[:, j // 32] >> (j % 32)) & 1) == 1

    def check(self):
        ok, x = self.allowed(), self.x.double()
        for r in range(self.m):
            ids = ok[r].nonzero()[:, 0]
            z = x[r, ids]
            n = min(self.k, z.numel())
            nan = torch.isnan(z)
            # a stable sort of the allowed entries, NaN after every number; the two zeros are equal
            order = torch.sort(torch.where(nan, torch.zeros_like(z), z), descending=True, stable=True).indices
            order = torch.cat((order[~nan[order]], nan.nonzero()[:, 0]))[:n]
            assert self.ids[r, :n].tolist() == ids[order].tolist(), f"row {r}"
            assert (self.ids[r, n:] == -1).all() and (self.top[r, n:] == -INF).all()
            tgt = int(self.target[r])
            scored = 0 <= tgt < self.v
            xt = float(x[r, tgt]) if scored and bool(ok[r, tgt]) else -INF
            if scored:
                want = 1 + int((~nan).sum() if math.isnan(xt) else (z > xt).sum())
                assert int(self.rank[r]) == want, f"row {r}"
            else:
                assert int(self.rank[r]) == (0 if tgt == -1 else -1)
                assert float(self.logprob[r]) == 0.0 if tgt == -1 else math.isnan(float(self.logprob[r]))
            if bool(nan.any()) or bool((z == INF).any()):
                assert torch.isnan(self.lse[r]) and torch.isnan(self.entropy[r]) and torch.isnan(self.top[r, :n]).all()
                assert not scored or torch.isnan(self.logprob[r])
                continue
            if z.numel() == 0 or float(z.max()) == -INF:
                assert float(self.lse[r]) == -INF and float(self.entropy[r]) == 0.0
                assert (self.top[r] == -INF).all() and (not scored or float(self.logprob[r]) == -INF)
                continue
            z = z / self.temp
            big = z.max()
            ls = (z - big).exp().sum().log()                       # around the largest: lse alone loses it at 10^38
            lse = big + ls
            p = (z - big - ls).exp()
            d = torch.where(p > 0, z - big, torch.zeros_like(z))
            ent = ls - (p * d).sum()
            # S: v/512 + 64 sums of positive terms at u each; an exponential is off by 4 u and by the rounding of its
            # argument, 3 u |z - M|, weighted by p; then the logarithm and the shift's own roundings
            es = U * (self.v / 512 + 64 + 4) + 3 * U * float((p * d.abs()).sum())
            tl = es + U * (2 * abs(float(lse)) + 2 * abs(float(big)) + 4)
            close(self.lse[r], lse, tl, f"lse {r}")
            te = 2 * es * (1 + float((p * d.abs()).sum())) + 3 * U * float((p * d * d).sum()) + U * (8 + 4 * abs(float(ent)))
            close(self.entropy[r], ent, te, f"entropy {r}")

            def near(got, val, what):
                if val == -INF:
                    assert float(got) == -INF
                    return
                w = torch.tensor(val / self.temp, dtype=torch.float64, device="cuda") - big - ls
                dz = abs(val / self.temp - float(big))
                close(got, w, es + U * (4 * dz + 2 * abs(float(w)) + 4 * abs(float(ls)) + 4), what)

            if scored:
                near(self.logprob[r], xt, f"logprob {r}")
            for i in range(n):
                near(self.top[r, i], float(x[r, ids[order[i]]]), f"top {r} {i}")


LP_CASES = [
    dict(m=1, v=1, k=1), dict(m=2, v=3, k=5), dict(m=3, v=31, k=32, mask=True), dict(m=2, v=33, k=0),
    dict(m=5, v=1000, k=20, temp=0.7, mask=True), dict(m=3, v=1025, k=3, t="bf16"), dict(m=4, v=4097, k=32, t="f16", pad=3),
    dict(m=1, v=131072, k=20, mask=True, temp=0.7), dict(m=1, v=50001, k=5, t="bf16"), dict(m=2, v=131072, k=32, t="f16"),
    dict(m=7, v=30000, k=1, off=1, t="bf16", pad=1), dict(m=9, v=30000, k=7, off=3, mask=True),
    dict(m=40, v=20001, k=5, t="bf16", temp=1.3), dict(m=64, v=9000, k=20, mask=True, pad=5),
    dict(m=200, v=5000, k=10), dict(m=200, v=5001, k=10, t="bf16", mask=True), dict(m=600, v=700, k=4, t="f16"),
    dict(m=2, v=600000, k=20), dict(m=1, v=2000001, k=8, t="bf16", mask=True),
    dict(m=3, v=8192, k=20, spread=60.0), dict(m=3, v=8192, k=20, spread=0.01, t="bf16"),
]


@pytest.mark.parametrize("c", LP_CASES, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_logprob_against_64_bits(Q, c):
    t = Lp(Q, seed=c["m"] + c["v"], **c)
    t.call()
    t.check()


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("v", [64, 5000, 70000])
def test_logprob_orders_that_are_hard_to_select_from(Q, t, v):
    """ascending, descending and constant rows, blocks of equal values, the two zeros, lowest values"""
    j = torch.arange(v, device="cuda", dtype=torch.float32)
    rows = [j / v, -j / v, torch.zeros(v, device="cuda"), (j % 7), -(j % 2) * 0.0 - 0.0, -(j // 100), -INF + 0 * j]
    rows.append(torch.where(j % 3 == 0, -INF, -j / v))
    rows.append(torch.where(j == v - 1, 50.0, torch.finfo(T[t]).min))
    rows.append(torch.full((v,), torch.finfo(T[t]).min, device="cuda"))
    rows.append(torch.where(j % 2 == 0, 0.0, -0.0) + 0 * j)
    logits = torch.stack(rows)
    for mask in (False, True):
        c = Lp(Q, len(rows), v, t, 20, mask=mask, pad=1, seed=v, logits=logits)
        c.call()
        c.check()


@pytest.mark.parametrize("m,v", [(8, 3000), (8, 40000), (400, 3000)])
def test_logprob_masked_empty_and_unscored_rows(Q, m, v):
    c = Lp(Q, m, v, "f32", 6, mask=True, pad=2, seed=9)
    ok = c.allowed()
    c.x[~ok] = torch.tensor([NAN, INF, -INF, torch.finfo(torch.float32).min], device="cuda")[
        torch.randint(0, 4, (int((~ok).sum()),), device="cuda", generator=gen(1))]
    c.bits[0] = 0                                                  # nothing allowed
    c.bits[1] = 0
    c.bits[1, 3] = 1 << 5                                          # one entry
    c.target[1] = 3 * 32 + 5
    c.x[1, 3 * 32 + 5] = -4.0
    c.bits[2, :-2] = 0                                             # only bits past the vocabulary, and a few
    c.x[3, c.allowed()[3]] = -INF                                  # allowed, but all -inf
    c.target[4] = -1
    c.target[5] = v
    c.target[6] = int((~c.allowed()[6]).nonzero()[0, 0])           # a masked target
    c.x[2, c.allowed()[2]] = 1.5
    c.call()
    c.check()


@pytest.mark.parametrize("m,v", [(7, 3000), (7, 70000), (400, 3000)])
def test_logprob_nan_and_inf(Q, m, v):
    c = Lp(Q, m, v, "f32", 8, seed=10)
    c.x[0, v // 2] = NAN
    c.x[1, 5] = INF
    c.x[2, 7] = -INF
    c.x[3] = NAN
    c.x[4, 11] = NAN
    c.target[4] = 11                                               # a NaN target
    c.x[5] = -INF
    c.x[5, 9] = NAN                                                # -inf and one NaN
    c.x[6] = torch.where(torch.arange(v, device="cuda") < v - 3, NAN, 1.0)   # three numbers, fewer than top_k
    c.call()
    c.check()


def test_logprob_outputs_may_be_left_out(Q):
    c = Lp(Q, 4, 5000, "f32", 3, seed=3)
    c.call()
    full = [t.clone() for t in (c.logprob, c.rank, c.lse, c.entropy, c.top, c.ids)]
    for name, want in (("logprob", full[0]), ("rank", full[1]), ("lse", full[2]), ("entropy", full[3])):
        for t in (c.logprob, c.lse, c.entropy, c.rank):
            t.fill_(5)
        others = {k: None for k in ("logprob", "rank", "lse", "entropy") if k != name}
        c.call(**others, **({"target": None} if name in ("lse", "entropy") else {}))
        assert torch.equal(getattr(c, name), want)
        for k in others:
            assert (getattr(c, k) == 5).all()
        assert torch.equal(c.top, full[4]) and torch.equal(c.ids, full[5])


def test_logprob_repeats_bit_for_bit_on_another_stream_and_in_a_graph(Q):
    for m, v, t in ((1, 131072, "f32"), (3, 50001, "bf16"), (500, 5000, "f32")):
        c = Lp(Q, m, v, t, 20, seed=8)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        c.call(stream=s)
        s.synchronize()
        outs = (c.logprob, c.rank, c.lse, c.entropy, c.top, c.ids)
        first = [o.clone() for o in outs]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            c.call(stream=s)
        for _ in range(10):
            for o in outs:
                o.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, first))


def test_logprob_of_large_offsets(Q):
    """the same distribution on logits around 10^4: the differences are exact in f32"""
    v = 4096
    base = torch.randint(-64, 64, (2, v), device="cuda", generator=gen(1)).float() / 8
    c = Lp(Q, 2, v, "f32", 4, logits=base)
    c.call()
    d = Lp(Q, 2, v, "f32", 4, logits=base + 8192.0)
    d.target.copy_(c.target)
    d.call()
    d.check()
    for a, b in ((c.logprob, d.logprob), (c.entropy, d.entropy), (c.top, d.top)):
        assert torch.equal(a, b)

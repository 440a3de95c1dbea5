"""The operators around the MoE layer on the GPU where their work is walked
through in parts: several tiles a block, ranges and places at the ends of what
the calls take.  Tolerances as in test_gpu_ops.py."""
import pytest
import torch
from test_gpu_ops import INF, U, Lp, Norm, Q, Q4, gen  # noqa: F401

pytestmark = pytest.mark.gpu


# 313 row tiles of 128 and one or two token tiles, more than there are SMs: blocks walk through several tiles.  Token
# tiles end below and above 128; rows end inside a stage, a group, and after odd numbers of groups.
@pytest.mark.parametrize("m", [100, 130, 300, 390, 512])
@pytest.mark.parametrize("k,group", [(352, 128), (160, 64), (96, 64), (352, 32), (160, 32), (1056, 128)])
def test_q4_many_tiles_a_block(Q, m, k, group):  # noqa: F811
    t = Q4(Q, m, 40001, k, group, zeros=True, x="bf16" if m % 4 else "f16", pado=3, seed=m + k + group)
    t.call()
    t.check()
    first = t.out.clone()
    for _ in range(3):
        t.out.zero_()
        t.call()
        assert torch.equal(t.out, first)


@pytest.mark.parametrize("m,v", [(3, 3001), (2, 70000), (400, 3000)])
@pytest.mark.parametrize("temp", [1e-36, 1e-20, 1e20, 5e28, 1e30, 1e36])
def test_logprob_far_temperatures(Q, temp, m, v):  # noqa: F811
    """logits of the temperature's own size; what is masked or -inf has no weight at any temperature"""
    rnd = torch.randn((m, v), device="cuda", generator=gen(v))
    for mask in (False, True):
        c = Lp(Q, m, v, "f32", 5, temp=temp, mask=mask, seed=m + v, logits=rnd * temp)
        c.x[0, 1::3] = -INF
        c.target[1] = 0
        c.x[1, 7] = -3e38                                          # far below at every temperature, and finite
        if mask:
            c.x[~c.allowed()] = torch.finfo(torch.float32).min
        c.call()
        c.check()


def test_logprob_entropy_of_a_far_largest_entry(Q):  # noqa: F811
    """sums of 10^9 around a reference 10^30 below the largest entry: their weight is zero"""
    v = 1 << 26
    c = Lp(Q, 1, 8, "f32", 1)
    c.v, c.cfg = v, Q.make_logprob_cfg(v, Q.MOE_T_F32, 1)
    c.x = torch.full((1, v), 5.0, device="cuda")
    c.x.view(-1, 1 << 16)[:, :1 << 14] = 0.0                       # lower references than most entries
    c.x[0, v - 5] = 2e30
    c.target[0] = v - 5
    c.call()
    assert int(c.ids[0, 0]) == v - 5 and int(c.rank[0]) == 1
    assert float(c.entropy[0]) == 0.0 and float(c.logprob[0]) == 0.0 and float(c.lse[0]) == float(c.x[0, v - 5])


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("m,n,k,group", [(1, 300, 5120, 128), (3, 64, 512, 32), (8, 1000, 2336, 64), (1, 40, 32768, 32),
                                         (40, 300, 512, 128)])
def test_q4_large_x_at_codes_equal_to_their_zero(Q, m, n, k, group, zeros):  # noqa: F811
    """x of 2^30 whose codes are the zeros, among small whole numbers: every sum is a whole number below 2^24, exact"""
    t = Q4(Q, m, n, k, group, zeros=zeros, seed=k + m)
    t.scales.fill_(1.0)
    t.x.copy_(torch.randint(-3, 4, (m, k), device="cuda", generator=gen(2)))
    for at in (5, k // 2, k - 1):                                  # even and odd codes
        t.x[:, at] = 2.0 ** 30
        z = t.zeros[:, at // group] if zeros else torch.full((n,), 8, dtype=torch.uint8, device="cuda")
        b = t.w[:, at // 2]
        t.w[:, at // 2] = (b & 0x0F) | (z << 4) if at & 1 else (b & 0xF0) | z
    t.call()
    assert torch.equal(t.out.double(), t.x.double() @ t.weights().t())


@pytest.mark.parametrize("m", [1, 8])
def test_q4_x_near_the_end_of_bf16(Q, m):  # noqa: F811
    """neighbours of one sign whose plain sum overflows f32, under small scales"""
    t = Q4(Q, m, 70, 512, 64, zeros=True, seed=4)
    t.scales.fill_(2.0 ** -12)
    t.x.fill_(2.0 ** 126)
    t.w[:] = 0x33
    t.zeros[:] = (torch.arange(70, device="cuda") % 3 + 1).to(torch.uint8)[:, None]
    t.call()
    want = t.x.double() @ t.weights().t()                          # 512 2^126 2^-12 times 2, 1 or 0: powers of two
    assert torch.equal(t.out.double(), want) and (want < 2.0 ** 125).all()


def range_mask(c, lo, hi):
    """allows the entries lo .. hi - 1 of every row"""
    j = torch.arange(c.bits.shape[1] * 32, device="cuda")
    on = ((j >= lo) & (j < hi)).view(-1, 32).long() << torch.arange(32, device="cuda")
    c.bits[:] = on.sum(1).to(torch.int32)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("m,v,lo,hi", [(3, 131072, 0, 5000), (2, 131072, 40000, 40007), (40, 70000, 0, 35001),
                                       (610, 9000, 100, 1500), (2, 9000, 8999, 9000), (310, 131072, 0, 65536)])
def test_logprob_of_a_range_of_the_vocabulary(Q, t, m, v, lo, hi):  # noqa: F811
    """masks that leave most warps and pieces nothing, over rows that rise, fall, or hold few values"""
    j = torch.arange(v, device="cuda", dtype=torch.float32)
    rows = torch.stack((j / v * 8, -j / v * 8, torch.zeros_like(j), j % 5, torch.full_like(j, -INF)))
    c = Lp(Q, m, v, t, 20, mask=True, pad=1, logits=rows[torch.arange(m, device="cuda") % 5])
    range_mask(c, lo, hi)
    c.call()
    if m > 40:                                                     # the check goes row by row
        first = [o.clone() for o in (c.logprob, c.lse, c.entropy, c.top, c.rank, c.ids)]
        assert all(torch.equal(c.ids[k], c.ids[k % 5]) for k in range(5, m))   # rows repeat but for their targets
        c.m, c.x, c.bits = 10, c.x[-10:], c.bits[-10:]
        c.target, c.logprob, c.lse, c.entropy, c.top, c.rank, c.ids = [c.target[-10:]] + [o[-10:] for o in first]
    c.check()


def test_logprob_of_a_range_takes_one_more_pass_not_many(Q):  # noqa: F811
    """rising rows of which half is allowed: without top entries about 50 us, with them a pass over the allowed half
    (an entry a thread at a time, 256 steps of about a microsecond, two rows a block) at the most"""
    m, v = 512, 131072
    c = Lp(Q, m, v, "f32", 20, mask=True, logits=torch.arange(v, device="cuda", dtype=torch.float32).expand(m, v) / v)
    range_mask(c, 0, v // 2)
    c.call()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    begin.record()
    c.call()
    end.record()
    torch.cuda.synchronize()
    assert c.ids[m // 2].tolist() == list(range(v // 2 - 1, v // 2 - 21, -1))
    assert begin.elapsed_time(end) < 5.0


@pytest.mark.parametrize("c", [
    dict(m=700, dim=7168, y="f32", h="f32"), dict(m=153, dim=8192, y="f32", h="f32", x="f32"),
    dict(m=500, dim=8192, y="f32", h="f32", post="layer", pre="layer", bias=True, gate="row", group=7),
    dict(m=310, dim=6880, y="f32", h="f32", gate="token", gt="bf16", group=3), dict(m=400, dim=8192, y="f32", h="bf16"),
    dict(m=900, dim=2304, post="layer", pre="layer", bias=True, gate="row", group=64, y="bf16", w="bf16"),
    dict(m=1300, dim=1024, bias=True, gate="row", gt="bf16", group=1, pad=8, h="f32", x="f16"),
], ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_norm_streamed_rows(Q, c):  # noqa: F811
    """more rows than blocks fit at once: the widest rows, and what is loaded beside a row (gate rows, biases)"""
    t = Norm(Q, seed=c["m"] + c["dim"], **c)
    t.call()
    t.check()
    want = t.h_out.clone(), t.x_out.clone()
    t.call(h_out=t.h)                                              # in place
    assert torch.equal(t.h, want[0]) and torch.equal(t.x_out, want[1])


@pytest.mark.parametrize("t,m,v", [("bf16", 700, 100741), ("f32", 700, 20001), ("f32", 400, 131072), ("f16", 1300, 6000)])
def test_logprob_of_equal_entries_in_many_rows(Q, t, m, v):  # noqa: F811
    """more equal entries than the candidate buffer takes, in every block's rows one after the other: the lowest ids"""
    c = Lp(Q, m, v, t, 5, pad=8, logits=torch.full((m, v), 1.5))
    for _ in range(5):
        c.ids.fill_(7)
        c.call()
        assert torch.equal(c.ids, torch.arange(5, dtype=torch.int32, device="cuda").expand(m, 5))
        assert (c.rank == 1).all() and (c.top == c.top[0, 0]).all()


@pytest.mark.parametrize("group", [128, 64, 32])
def test_q4_many_tokens_with_cold_zeros(Q, group):  # noqa: F811
    """long rows whose weights, scales and zeros come from memory: the dequantising warps wait for zeros while the copies
    run ahead, and may not be overtaken by them"""
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for i, (m, n, k, x) in enumerate([(128, 3372, 26784, "bf16"), (64, 2193, 21056, "bf16"), (256, 1537, 27008, "f16"),
                                      (172, 3268, 28352, "f16"), (73, 20744, 10560, "bf16"), (71, 40030, 7456, "f16")]):
        t = Q4(Q, m, n, k, group, zeros=True, x=x, seed=i)
        want = t.x.double() @ t.weights().t()
        for _ in range(30):
            flush.fill_(i)
            t.call()
            assert (t.out.double() - want).norm() / want.norm() <= 2 * U * max(32, k / 16), (m, n, k)

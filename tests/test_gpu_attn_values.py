"""That no key's value is left out of attention over the cache, and its error in norm.

With random values of either sign a sum is as small as its largest terms' root of squares, and a bound in
sum p |v| lets a kernel pass that drops a tile of a long context.  Here keys of zero make every weight
one and values count: slot j holds a one at value j of the head (modulo its width) in one of a few passes, and
zeros in the others, so that a value of the output is a count of at most COUNT slots over the number of keys seen.
u is half a step of the cache's type.
"""
import pytest
import torch
from test_gpu_attn import Attn, Q  # noqa: F401
from test_gpu_ops import INF, NAN, U, half_step

COUNT = 60   # one slot more or less is 1 / 60, 4 half steps of bf16


def passes(length, dim):
    return max(1, -(-length // (COUNT * dim)))


def values(length, dim, head, n, of, device):
    """[length, dim] of zeros and ones; a slot has its one in one of the passes"""
    j = torch.arange(length, device=device)
    v = torch.zeros((length, dim), device=device)
    v[j, (j + 5 * head) % dim] = ((j // dim) % of == n).float()
    return v


def counts(seen, v):
    """ones that each token sees, and keys"""
    count = (seen.float() @ v).double()
    assert count.max() <= COUNT
    return count, seen.double().sum(1, keepdim=True)


def wrong(got, count, keys, t):
    """where an output is not the mean of what its token sees: sums of ones are exact in f32; a reciprocal, a product
    and the output's rounding"""
    want = torch.where(keys > 0, count / keys.clamp(min=1), 0.0)
    return (got.double() - want).abs() > half_step(t, want) * (1 + 2.0 ** -10) + 4 * U * want


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("length,dim", [(700, 64), (20000, 128), (20000, 64), (50000, 128)])
def test_a_lost_slot_is_seen(length, dim, t):
    """the check itself, without a GPU: an oracle that leaves out one slot, or one slot's value"""
    g = torch.Generator().manual_seed(length)
    seen = torch.ones((1, length), dtype=torch.bool)
    kind = torch.bfloat16 if t == "bf16" else torch.float16
    of = passes(length, dim)
    lost = [0, 31, 32, 127, length - 1, *torch.randint(0, length, (5,), generator=g).tolist()]
    found = [0] * len(lost)
    for n in range(of):
        v = values(length, dim, 3, n, of, "cpu")
        count, keys = counts(seen, v)
        assert not wrong((count / keys).to(kind), count, keys, t).any()
        for i, j in enumerate(lost):
            found[i] += int(wrong(((count - v[j]) / keys).to(kind), count, keys, t).any())
    assert found == [1] * len(lost)


@pytest.mark.gpu
@pytest.mark.parametrize("max_new", [1, 5000])
@pytest.mark.parametrize("c", [
    dict(new=[1], kv=[20000], heads=8, kv_heads=1, dim=128, page=16),
    dict(new=[1, 3, 1], kv=[131000, 700, 4097], heads=8, kv_heads=4, dim=128, page=64),
    dict(new=[1] * 20, kv=[100 + 333 * i for i in range(20)], heads=6, kv_heads=2, dim=64, page=32, t="f16", order="hnd"),
    dict(new=[300], kv=[9000], heads=4, kv_heads=1, dim=128, page=16),
    dict(new=[70, 200], kv=[20000, 200], heads=7, kv_heads=1, dim=64, page=8, t="f16"),
    dict(new=[150], kv=[6000], heads=12, kv_heads=2, dim=96, page=32, window=1001),
    dict(new=[33, 150], kv=[3000, 777], heads=4, kv_heads=2, dim=80, page=128, causal=False),
], ids=["one-20000", "long-131000", "many-of-64", "chunk", "seven-heads", "window", "cross"])
def test_every_slot_reaches_the_output(Q, c, max_new):  # noqa: F811
    a = Attn(Q, max_new=max_new, **c)
    a.k.zero_()
    a.v.zero_()
    a.spoil(INF)
    of, group = passes(max(a.kv), a.dim), a.heads // a.kv_heads
    where = [a.slots(b) for b in range(a.batch)]
    seen = [a.visible(b) for b in range(a.batch)]
    for n in range(of):
        held = [[values(a.kv[b], a.dim, h, n, of, "cuda") for h in range(a.kv_heads)] for b in range(a.batch)]
        for b in range(a.batch):
            for h in range(a.kv_heads):
                a.v[where[b][0], where[b][1], h] = held[b][h].to(a.v.dtype)
        a.out.fill_(NAN)
        a.call()
        out = a.out.view(a.m, a.heads, a.dim)
        for b in range(a.batch):
            for h in range(a.heads):
                bad = wrong(out[a.cu[b]:a.cu[b + 1], h], *counts(seen[b], held[b][h // group]), a.t)
                assert not bad.any(), (n, b, h, bad.nonzero()[:3].tolist())
    assert Q.moe_v41_read_status(a.ws) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("max_new", [1, 5000])
@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("c", [
    dict(new=[1], kv=[700], heads=16, kv_heads=2, dim=128, page=16),
    dict(new=[1], kv=[20000], heads=16, kv_heads=2, dim=128, page=16),
    dict(new=[2], kv=[200000], heads=8, kv_heads=1, dim=64, page=64),
    dict(new=[100], kv=[9000], heads=4, kv_heads=1, dim=128, page=32),
], ids=["700", "20000", "200000", "chunk"])
def test_the_error_in_norm(Q, c, t, max_new):  # noqa: F811
    """Weights are off by at most u, in either direction and each on its own, so that the square of a head's error is
    about u^2 / 3 sum p^2 v^2 and at most four times u^2 of it over 64 values and more; scores by e (as derived in
    Attn.check), likewise; sums of f32 by two U of what has been summed up a step, which is of the size of their
    result; and the output by u."""
    u = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}[t]
    a = Attn(Q, t=t, max_new=max_new, seed=3, **c)
    a.call()
    group, (page, slot), seen = a.heads // a.kv_heads, a.slots(0), a.visible(0)
    out = a.out.view(a.m, a.heads, a.dim).double()
    for h in range(a.heads):
        k, v = (x[page, slot, h // group].double() for x in (a.k, a.v))
        q = a.q.view(a.m, a.heads, a.dim)[:, h].double()
        s = ((q @ k.t()) * a.scale).masked_fill(~seen, -INF)
        p = torch.softmax(s, -1)
        want, root = p @ v, ((p * p) @ (v * v)).sum(-1).sqrt()
        e = 2 * U * (a.dim + 8) * (q.abs().amax(-1) * k.abs().sum(-1).max()).max() * a.scale \
            + 8 * U * s.masked_fill(~seen, 0.0).abs().max() + 2.0 ** -20
        size = want.norm(dim=-1)
        sums = 2 * U * (a.kv[0] / 16 + 64)
        tol = (2 * u + 2 * e) * root + 1.01 * u * size + sums * (root + size)
        gap = (out[:, h] - want).norm(dim=-1)
        assert (gap <= tol).all(), (h, (gap / tol).max().item())
        # over all rows (one whose weights are few and large has a large output and bound) that is less than what a
        # tile of 32 keys adds, the root of its share
        assert a.kv[0] > 20000 or tol.norm() < (32 / a.kv[0]) ** 0.5 * size.norm()

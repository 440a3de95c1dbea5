"""The scoring example's step on the GPU: each operator's output against 64-bit
torch from what the operator was given, and a graph replay against the first run.

u = 2^-24 is half a step of f32, 2^-8 of bf16 (relative to the value).
"""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def scorer():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "score_tokens.py")
    spec = importlib.util.spec_from_file_location("score_tokens", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    s = mod.Scorer(mod.W.WORKLOADS["tiny"], layers=2, vocab=1000, top_k=5)
    s.step()
    torch.cuda.synchronize()
    s.check_status()
    return s


def rms(v, w):
    return v / ((v * v).mean(1, keepdim=True) + 1e-6).sqrt() * w.double()


def test_norms(scorer):
    s = scorer
    # the mean square (at most 64 sums in a row), root and products: under 72 roundings of u each, 2^-17 in all; the
    # residual sum adds two of its terms' sizes, and x passes on what h was off by (itself, and through its scale)
    x0 = rms(s.h[0].double(), s.pre_w[0])
    assert ((s.x[0].double() - x0).abs() <= (2.0 ** -17 + 2.0 ** -8) * 1.001 * x0.abs()).all()
    for i in range(len(s.layers)):
        h, n = s.h[i].double(), rms(s.y[i].double(), s.post_w[i])
        th = 2.0 ** -17 * n.abs() + 4 * U * (h.abs() + n.abs())
        assert ((s.h[i + 1].double() - (h + n)).abs() <= th).all()
        x = rms(h + n, s.pre_w[i + 1])
        r = 1.0 / ((h + n).square().mean(1, keepdim=True)).sqrt()
        big = th.max(1, keepdim=True).values
        tx = 2.0 ** -17 * x.abs() + (s.pre_w[i + 1].double() * th + x.abs() * big) * r * 1.01
        assert ((s.x[i + 1].double() - x).abs() <= tx + 2.0 ** -8 * 1.001 * x.abs()).all()


def test_head_and_scores(scorer):
    s = scorer
    q = torch.stack((s.head & 15, s.head >> 4), -1).reshape(s.vocab, s.w.dim).double() - 8
    wt = q * s.scales.double().repeat_interleave(128, 1)[:, :s.w.dim]
    x = s.x[-1].double()
    # sums of dim products in any order, 2 u each, and the factor of a group
    tol = 2 * U * (s.w.dim + 64) * (x.abs() @ wt.abs().t())
    assert ((s.logits.double() - x @ wt.t()).abs() <= tol).all()

    # from the logits the kernel was given: lse, and what is taken off it, in f32 with sums of 1000 positive terms (at
    # most 64 in a row) and exponentials of 2 u relative error plus u |z - max| from their arguments
    z = s.logits.double()
    lse = torch.logsumexp(z, 1)
    span = (z.max(1).values - z.min(1).values).max()
    tol = U * (256 + 8 * float(span)) + 4 * U * float(z.abs().max())
    assert ((s.lse.double() - lse).abs() <= tol).all()
    zt = z.gather(1, s.target.long()[:, None])
    assert ((s.logprob.double() - (zt[:, 0] - lse)).abs() <= tol).all()
    assert torch.equal(s.rank.long(), 1 + (z > zt).sum(1))
    p = torch.softmax(z, 1)
    entropy = -(p * torch.log_softmax(z, 1)).sum(1)
    # the entropy's second sum carries terms of up to |z - max|
    assert ((s.entropy.double() - entropy).abs() <= tol * (2 + float(span))).all()
    order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :5]
    assert torch.equal(s.top_id.long(), order)
    assert ((s.top_logprob.double() - (z.gather(1, order) - lse[:, None])).abs() <= tol).all()


def test_graph_replay_gives_the_same(scorer):
    s = scorer
    want = [t.clone() for t in (s.logits, s.logprob, s.rank, s.entropy, s.top_logprob, s.top_id)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        s.step()
    for t in (s.logits, s.logprob, s.entropy, s.top_logprob):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    s.check_status()
    for a, b in zip(want, (s.logits, s.logprob, s.rank, s.entropy, s.top_logprob, s.top_id)):
        assert torch.equal(a, b)

"""The attention block's operators as programs use them: calls at once on two streams,
one workspace for calls of several kinds and for several graphs, sequences that share
pages, batches with many sequences that have nothing new, the limits of the arguments.
Outputs are compared with the same call alone (bit for bit) or with 64-bit torch."""
import pytest
import torch
from test_gpu_attn import Attn, Q, desc, gen  # noqa: F401

pytestmark = pytest.mark.gpu

FEW = dict(new=[1, 2, 1], kv=[30000, 4000, 17], heads=8, kv_heads=2, dim=128, page=16)
MANY = dict(new=[400, 3, 200], kv=[6000, 900, 200], heads=12, kv_heads=2, dim=64, page=32, t="f16")


def test_two_calls_at_once(Q):  # noqa: F811
    """on two streams, each with its workspace, over one another"""
    calls = [Attn(Q, seed=1, **FEW), Attn(Q, seed=2, **MANY)]
    for a in calls:
        a.call()
        a.check()
        a.want = a.out.clone(), a.lse.clone()
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(20):
        for a, s in zip(calls, streams):
            with torch.cuda.stream(s):
                a.out.fill_(7.0)
                a.call()
    torch.cuda.synchronize()
    for a in calls:
        assert torch.equal(a.out[:a.cu[-1]], a.want[0][:a.cu[-1]]) and torch.equal(a.lse, a.want[1])
        assert Q.moe_v41_read_status(a.ws) == 0


def test_one_workspace_for_every_call_of_a_stream(Q):  # noqa: F811
    """both kernels, other head sizes, types and cuts, one after another and in two graphs"""
    calls = [Attn(Q, seed=i, **c) for i, c in enumerate((FEW, MANY, dict(FEW, dim=64), dict(MANY, new=[1, 3, 2], dim=128)))]
    for a in calls:
        a.call()
        a.check()
        a.want = a.out.clone()
    ws = max((a.ws for a in calls), key=torch.numel)
    for a in calls:
        a.ws = ws
    graphs = []
    for order in (calls, calls[::-1]):
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            for a in order:
                a.call()
        graphs.append(graph)
    for graph in graphs * 3:
        for a in calls:
            a.out.zero_()
        graph.replay()
        for a in calls:
            assert torch.equal(a.out[:a.cu[-1]], a.want[:a.cu[-1]])
    assert Q.moe_v41_read_status(ws) == 0


@pytest.mark.parametrize("max_new", [1, 100])
def test_sequences_that_share_pages(Q, max_new):  # noqa: F811
    """a common prompt is stored once: the same pages in several rows of the table"""
    a = Attn(Q, [1, 5, 3], [1000, 1007, 990], 8, 2, 128, page=16, max_new=max_new)
    a.table[1:, :50] = a.table[0, :50]
    a.call()
    a.check()


@pytest.mark.parametrize("max_new", [1, 100])
def test_batches_with_sequences_that_have_nothing_new(Q, max_new):  # noqa: F811
    """more sequences than a block has threads, and mostly empty ones between and behind"""
    new = [0] * 5000
    kv = [0] * 5000
    for i, (n, k) in {0: (1, 40), 383: (2, 700), 384: (1, 9), 1900: (3, 2000), 4999: (1, 33)}.items():
        new[i], kv[i] = n, k
    a = Attn(Q, new, kv, 4, 2, 64, page=16, max_new=max_new)
    a.spoil(float("nan"))
    a.call()
    a.check()
    k = torch.randn((a.m, 2, 64), generator=gen(3), device="cuda").bfloat16()
    Q.moe_v41_kv_append(a.kv_cfg, Q.make_rope_cfg(64, 0), a.seqs, a.m, k, 128, k, 128, a.k, a.v, 0, None, 0, None, 0, None,
                        None, None)
    for b in (0, 383, 384, 1900, 4999):
        p, s = a.slots(b)
        assert torch.equal(a.v[p[-new[b]:], s[-new[b]:]], k[a.cu[b]:a.cu[b + 1]])


@pytest.mark.parametrize("c,max_new", [
    (dict(new=[1], kv=[100], heads=4096, kv_heads=1024, dim=16, page=8), 1),
    (dict(new=[2], kv=[300], heads=4096, kv_heads=1, dim=16, page=16), 2),          # 4096 heads share a key head
    (dict(new=[40], kv=[70], heads=1024, kv_heads=1024, dim=24, page=8), 40),
    (dict(new=[3] * 2000, kv=[3 + i % 40 for i in range(2000)], heads=2, kv_heads=1, dim=32, page=8), 3),
    (dict(new=[20] * 600, kv=[20 + i % 50 for i in range(600)], heads=2, kv_heads=1, dim=32, page=8, t="f16"), 20),
], ids=lambda c: desc(c)[:60] if isinstance(c, dict) else str(c))
def test_attention_at_the_limits_of_heads_and_sequences(Q, c, max_new):  # noqa: F811
    a = Attn(Q, max_new=max_new, **c)
    a.call()
    if len(a.new) <= 1:
        a.check()
    else:
        a.check(only=list(range(0, len(a.new), 37)) + [len(a.new) - 1])


@pytest.mark.parametrize("max_new", [1, 100])
def test_pitches_that_are_never_stepped_by(Q, max_new):  # noqa: F811
    """one page, one key head, one new token: what their pitches say has no influence"""
    a = Attn(Q, [1], [50], 4, 1, 64, page=64, extra_pages=0, max_new=max_new)
    a.kv_cfg = Q.make_kv_cfg(1, 64, 64, 1, a.kv_cfg.type, -5, 64, 3)
    a.cfg = Q.make_attn_cfg(a.kv_cfg, 4, True, 0, a.scale)
    Q.moe_v41_paged_attention(a.cfg, a.seqs, 1, max_new, a.q, 0, a.k, a.v, a.out, -8, a.lse, 0, a.ws)
    a.check()
    k = torch.randn((1, 1, 64), generator=gen(4), device="cuda").bfloat16()
    Q.moe_v41_kv_append(a.kv_cfg, Q.make_rope_cfg(64, 0), a.seqs, 1, k, 0, k, -1, a.k, a.v, 0, None, 0, None, 0, None, None,
                        None)
    assert torch.equal(a.k[0, 49], k[0]) and torch.equal(a.v[0, 49], k[0])


@pytest.mark.parametrize("max_new", [1, 5000])
def test_rows_past_m_are_left_out(Q, max_new):  # noqa: F811
    """cu_new reaches behind the rows of the call: those there are get what they would"""
    a = Attn(Q, [3, 60], [40, 300], 4, 2, 64, page=16, max_new=max_new)
    a.m = 20
    a.call()
    assert (a.out[20:] == 77.0).all() and (a.lse[20:] == 77.0).all()
    all_kv, a.new, a.kv, a.cu = a.kv, [3, 17], [40, 257], [0, 3, 20]          # what the first 20 rows are
    a.full, a.out = a.full[:20], a.out[:20]
    a.check()
    a.kv = all_kv
    keep = a.k.clone(), a.v.clone()
    k = torch.randn((63, 2, 64), generator=gen(5), device="cuda").bfloat16()
    Q.moe_v41_kv_append(a.kv_cfg, Q.make_rope_cfg(64, 0), a.seqs, 20, k, 128, k, 128, a.k, a.v, 0, None, 0, None, 0, None,
                        None, None)
    p, s = a.slots(1)
    keep[0][p[240:257], s[240:257]] = k[3:20]
    p, s = a.slots(0)
    keep[0][p[-3:], s[-3:]] = k[:3]
    assert torch.equal(a.k, keep[0])


@pytest.mark.parametrize("max_new", [1, 5000])
def test_lengths_far_off(Q, max_new):  # noqa: F811
    """far below zero and far above the table"""
    a = Attn(Q, [4, 4, 4, 4], [60, 60, 60, 60], 4, 2, 64, page=16, tail=2, max_new=max_new)
    a.ints[1].copy_(torch.tensor([-2 ** 31, 2 ** 31 - 1, 60, -1], dtype=torch.int32))
    a.call()
    assert Q.moe_v41_read_status(a.ws, clear=True) == Q.MOE_STATUS_BAD_PAGE
    assert (a.out[:4] == 0).all() and (a.out[12:16] == 0).all()
    a.check(only=[2])
    a.ints[1].copy_(torch.tensor(a.kv, dtype=torch.int32))
    a.call()
    a.check()                                                            # the workspace is ready for the next call

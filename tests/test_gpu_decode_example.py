"""The decoding example's step on the GPU: each operator's output against 64-bit torch
from what the operator was given, over several steps, and a graph replay of a run
against the same run without.

u = 2^-24 is half a step of f32, 2^-8 of bf16 (relative to the value).
"""
import importlib.util
import os

import pytest
import torch
from test_gpu_attn import rope_tol, turned

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
CONTEXTS = [5, 700, 0, 333]


@pytest.fixture(scope="module")
def mod():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_step.py")
    spec = importlib.util.spec_from_file_location("decode_step", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def decoder(mod, steps):
    return mod.Decoder(mod.W.WORKLOADS["tiny"], CONTEXTS, steps)


def weights(lin):
    q = torch.stack((lin.w & 15, lin.w >> 4), -1).reshape(lin.n, lin.k).double() - 8
    return q * lin.scales.double().repeat_interleave(128, 1)[:, :lin.k]


def test_every_operator_of_every_step(mod):
    steps = 20
    dec = decoder(mod, steps)
    H, KH, D = mod.HEADS, mod.KV_HEADS, mod.HEAD_DIM
    keys = [dec.k_cache.clone(), dec.v_cache.clone()]
    for i in range(steps):
        dec.step()
        torch.cuda.synchronize()
        dec.check_status()
        assert dec.kv_len.tolist() == [c + i + 1 for c in CONTEXTS]
        # projection: sums of 512 products in any order, 2 u each, and the output's rounding
        wt, x = weights(dec.qkv_w), dec.x_a.double()
        want = x @ wt.t()
        tol = 2 * U * (dec.w.dim + 64) * (x.abs() @ wt.abs().t()) + 2.0 ** -8 * 1.01 * want.abs()
        assert ((dec.qkv.double() - want).abs() <= tol).all()
        # rotation and append: this step's slots, and no others
        qkv = dec.qkv.view(dec.m, H + 2 * KH, D)
        pos = dec.kv_len.long() - 1
        for got, given in ((dec.q.view(dec.m, H, D), qkv[:, :H]),):
            w = turned(given, pos, dec.freqs, 0, 0)
            t = rope_tol(given, pos, dec.freqs, 0, 0, 1.0, "bf16") + 2.0 ** -8 * 1.01 * w.abs()
            assert ((got.double() - w).abs() <= t).all()
        page, slot = dec.table.long().gather(1, (pos // dec.page)[:, None])[:, 0], pos % dec.page
        w = turned(qkv[:, H:H + KH], pos, dec.freqs, 0, 0)
        t = rope_tol(qkv[:, H:H + KH], pos, dec.freqs, 0, 0, 1.0, "bf16") + 2.0 ** -8 * 1.01 * w.abs()
        assert ((dec.k_cache[page, slot].double() - w).abs() <= t).all()
        keys[0][page, slot], keys[1][page, slot] = dec.k_cache[page, slot], qkv[:, H + KH:]
        assert torch.equal(dec.k_cache, keys[0]) and torch.equal(dec.v_cache, keys[1])
        # attention of each sequence over its cache: weights rounded to bf16, then the output
        for b in range(dec.m):
            n = int(dec.kv_len[b])
            j = torch.arange(n, device="cuda")
            where = dec.table[b].long()[j // dec.page], j % dec.page
            for h in range(H):
                k, v = (c[where[0], where[1], h // (H // KH)].double() for c in (dec.k_cache, dec.v_cache))
                q = dec.q.view(dec.m, H, D)[b, h].double()
                s = k @ q * D ** -0.5
                p = torch.softmax(s, 0)
                want = p @ v
                e = 2 * U * (D + 8) * (k.abs() @ q.abs()).max() * D ** -0.5 + 8 * U * s.abs().max() + 2.0 ** -20
                tol = (2.0 ** -8 + 2 * e + 2 * U * (n / 16 + 64)) * (p @ v.abs()) + 2.0 ** -8 * 1.01 * want.abs()
                assert ((dec.a.view(dec.m, H, D)[b, h].double() - want).abs() <= tol).all()
        # output projection, residual
        wt, x = weights(dec.o_w), dec.a.double()
        tol = 2 * U * (H * D + 64) * (x.abs() @ wt.abs().t())
        assert ((dec.y_a.double() - x @ wt.t()).abs() <= tol).all()
        h = dec.h.double() + dec.y_a.double()
        assert ((dec.h_mid.double() - h).abs() <= 4 * U * (dec.h.double().abs() + dec.y_a.double().abs())).all()
        # the norm after the experts: under 72 roundings of u, 2^-17 in all, and the sum's
        y = dec.y_f.double()
        n = y / ((y * y).mean(1, keepdim=True) + 1e-6).sqrt() * dec.norm_y.double()
        tol = 2.0 ** -17 * n.abs() + 4 * U * (dec.h_mid.double().abs() + n.abs())
        assert ((dec.next_h.double() - (dec.h_mid.double() + n)).abs() <= tol).all()
        dec.h.copy_(dec.next_h)


def test_graph_replay_gives_the_same(mod):
    steps = 12
    one, two = decoder(mod, steps + 1), decoder(mod, steps + 1)
    for _ in range(steps):
        one.step()
        one.h.copy_(one.next_h)
    two.step()                                                        # loads what a capture may not
    two.kv_len -= 1
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        two.step()
        two.h.copy_(two.next_h)
    for _ in range(steps):
        graph.replay()
    torch.cuda.synchronize()
    for d in (one, two):
        d.check_status()
    assert torch.equal(one.kv_len, two.kv_len) and torch.isfinite(one.h).all()
    for a, b in ((one.h, two.h), (one.k_cache, two.k_cache), (one.v_cache, two.v_cache), (one.a, two.a), (one.top_i, two.top_i)):
        assert torch.equal(a, b)

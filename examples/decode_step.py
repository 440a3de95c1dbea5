"""Decode tokens with a block of attention and quantized experts over a paged cache.

    python examples/decode_step.py [--steps 32] [--page 16]

Every step takes one token of each sequence through

    x = N(h)                                          moe_v41_block_norm (no block output yet)
    q, k, v = W4 x                                    moe_v41_q4_linear
    rotate q and k, store k and v in the cache        moe_v41_kv_append
    a = attention of q over the cache                 moe_v41_paged_attention
    y = W4 a;  h += y;  x = N(h)                      moe_v41_q4_linear, moe_v41_block_norm
    y = MoE(x);  h += N(y)                            moe_v41_forward, moe_v41_block_norm

Weights and inputs are synthetic, the block's output is the next step's input.  The
lengths live on the device and grow with every step, so that one captured graph
serves them all (main replays it and times it).
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import quantized_mixture_experts_router_gb300 as Q  # noqa: E402
import synth.workloads as W  # noqa: E402
from synth.device import stage_layer  # noqa: E402

HEADS, KV_HEADS, HEAD_DIM, GROUP = 8, 2, 64, 128


class Linear4:
    """a 4-bit weight [n, k] with its workspace"""

    def __init__(self, n, k, m, out_type, g, device):
        self.n, self.k = n, k
        self.w = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8, device=device)
        self.scales = ((torch.rand((n, -(-k // GROUP)), generator=g, device=device) + 0.5) / (4.6 * math.sqrt(k))).half()
        self.cfg = Q.make_q4_cfg(n, k, GROUP, out_type=out_type, max_tokens=m)
        self.ws = torch.empty(Q.moe_v41_q4_workspace_bytes(self.cfg), dtype=torch.uint8, device=device)
        Q.moe_v41_workspace_init(self.ws)

    def __call__(self, x, m, out):
        Q.moe_v41_q4_linear(self.cfg, x, m, self.k, self.w, self.scales, None, out, self.n, self.ws)


class Decoder:
    def __init__(self, w, contexts, steps, page=16, seed=0, device="cuda:0"):
        """contexts: tokens that each sequence has before the first step"""
        g = torch.Generator(device=device).manual_seed(seed)
        m, d = len(contexts), w.dim
        self.w, self.m, self.page = w, m, page

        def empty(*shape, dtype=torch.float32):
            return torch.empty(shape, dtype=dtype, device=device)

        def norm_weight():
            return torch.rand((d,), generator=g, device=device) + 0.5

        # the cache: pages of every sequence, in any order, filled as if its context had been read
        need = [-(-(c + steps) // page) for c in contexts]
        self.n_pages = sum(need)
        order = torch.randperm(self.n_pages, generator=g, device=device).int()
        self.table = torch.full((m, max(need)), -1, dtype=torch.int32, device=device)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (self.n_pages, page, KV_HEADS, HEAD_DIM)
        self.k_cache, self.v_cache = (torch.randn(shape, generator=g, device=device).bfloat16() for _ in range(2))
        self.kv_cfg = Q.make_kv_cfg(KV_HEADS, HEAD_DIM, page, self.n_pages)
        self.cu_new = torch.arange(m + 1, dtype=torch.int32, device=device)
        self.kv_len = torch.tensor(contexts, dtype=torch.int32, device=device)
        self.seqs = Q.make_seqs(m, self.cu_new, self.kv_len, self.table, self.table.shape[1])

        # attention: projections of 4 bits, rotation of the whole head
        row = (HEADS + 2 * KV_HEADS) * HEAD_DIM
        self.qkv_w = Linear4(row, d, m, Q.MOE_T_BF16, g, device)
        self.o_w = Linear4(d, HEADS * HEAD_DIM, m, Q.MOE_T_F32, g, device)
        freqs, magnitude = Q.moe_v41_rope_freqs(HEAD_DIM)
        self.freqs = torch.tensor(freqs, dtype=torch.float64, device=device)
        self.rope = Q.make_rope_cfg(HEAD_DIM, magnitude=magnitude)
        self.attn = Q.make_attn_cfg(self.kv_cfg, HEADS, scale=HEAD_DIM ** -0.5)
        self.attn_ws = empty(Q.moe_v41_attn_workspace_bytes(self.attn), dtype=torch.uint8)
        Q.moe_v41_workspace_init(self.attn_ws)
        self.qkv = empty(m, row, dtype=torch.bfloat16)
        self.q, self.a = (empty(m, HEADS * HEAD_DIM, dtype=torch.bfloat16) for _ in range(2))

        # experts
        self.layer = stage_layer(w.with_(m=m), 0, device=device, experts_on_gpu=True)
        self.moe = Q.make_cfg(w.dim, w.inter, w.n_routed, w.topk, w.gate_temp, w.norm_topk_prob, w.route_scale,
                              w.swiglu_limit, max_tokens=m)
        self.moe_ws = empty(Q.moe_v41_workspace_bytes(self.moe), dtype=torch.uint8)
        Q.moe_v41_workspace_init(self.moe_ws)
        self.top_w, self.top_i = empty(m, w.topk), empty(m, w.topk, dtype=torch.int32)

        # the norms between: f32 block outputs and stream, bf16 block inputs
        self.norm = Q.make_norm_cfg(d, Q.MOE_NORM_NONE, Q.MOE_NORM_RMS, Q.MOE_T_F32, Q.MOE_T_F32)
        self.last = Q.make_norm_cfg(d, Q.MOE_NORM_RMS, Q.MOE_NORM_NONE, Q.MOE_T_F32, Q.MOE_T_F32)
        self.norm_a, self.norm_f, self.norm_y = (norm_weight() for _ in range(3))
        self.h = torch.randn((m, d), generator=g, device=device)
        self.h_mid = empty(m, d)
        self.x_a, self.x_f = (empty(m, d, dtype=torch.bfloat16) for _ in range(2))
        self.y_a, self.y_f = empty(m, d), empty(m, d)
        self.next_h = empty(m, d)
        Q.moe_v41_block_norm(self.norm, m, None, 0, None, None, None, 0, self.h, d, None, 0, self.norm_a, None, self.x_a, d)

    def step(self):
        """kernels on the current stream alone; self.next_h is what the next step's h would be"""
        m, d, hd, row = self.m, self.w.dim, HEAD_DIM, self.qkv.shape[1]
        k, v = self.qkv[:, HEADS * hd:], self.qkv[:, (HEADS + KV_HEADS) * hd:]
        self.kv_len += 1
        Q.moe_v41_block_norm(self.norm, m, None, 0, None, None, None, 0, self.h, d, None, 0, self.norm_a, None,
                             self.x_a, d)
        self.qkv_w(self.x_a, m, self.qkv)
        Q.moe_v41_kv_append(self.kv_cfg, self.rope, self.seqs, m, k, row, v, row, self.k_cache, self.v_cache, HEADS,
                            self.qkv, row, self.q, HEADS * hd, self.freqs, None, None)
        Q.moe_v41_paged_attention(self.attn, self.seqs, m, 1, self.q, HEADS * hd, self.k_cache, self.v_cache, self.a,
                                  HEADS * hd, None, 0, self.attn_ws)
        self.o_w(self.a, m, self.y_a)
        Q.moe_v41_block_norm(self.norm, m, self.y_a, d, None, None, None, 0, self.h, d, self.h_mid, d, self.norm_f,
                             None, self.x_f, d)
        dl = self.layer
        Q.moe_v41_forward(self.moe, self.x_f, m, dl.router_w, dl.bias, dl.expert_ptrs, self.w.shared_kind, dl.sh1,
                          dl.sh3, dl.sh2, self.y_f, self.top_w, self.top_i, None, self.moe_ws)
        Q.moe_v41_block_norm(self.last, m, self.y_f, d, self.norm_y, None, None, 0, self.h_mid, d, self.next_h, d, None,
                             None, None, 0)

    def check_status(self):
        for ws in (self.attn_ws, self.moe_ws, self.qkv_w.ws, self.o_w.ws):
            status = Q.moe_v41_read_status(ws)
            if status:
                raise RuntimeError(f"device status {status}")


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--steps", type=int, default=32)
    p.add_argument("--page", type=int, default=16)
    a = p.parse_args()
    torch.cuda.set_device(0)
    contexts = [5, 700, 64, 333]
    dec = Decoder(W.WORKLOADS["tiny"], contexts, a.steps + 1, a.page)
    dec.step()
    dec.h.copy_(dec.next_h)
    torch.cuda.synchronize()
    dec.check_status()

    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        dec.step()
        dec.h.copy_(dec.next_h)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    dec.check_status()
    print(f"lengths {contexts} -> {dec.kv_len.tolist()}, |h| {float(dec.h.norm()):.3f}")
    print(f"{begin.elapsed_time(end) / a.steps * 1e3:.1f} us a step of {dec.m} sequences (graph replay)")


if __name__ == "__main__":
    main()

"""Score tokens with a small stack of quantized MoE layers.

    python examples/score_tokens.py [--layers 2] [--vocab 1000] [--top 5]

Hidden states go through `layers` MoE feed-forward blocks, each between its
norms, then through a 4-bit output head, and every token's target gets its log
probability, rank and the likeliest alternatives:

    x = N_pre(h)                                     moe_v41_block_norm (no block output yet)
    y = MoE(x);  h += N_post(y);  x = N_pre'(h)      moe_v41_forward, moe_v41_block_norm
    logits = W4 x                                    moe_v41_q4_linear
    log p(target), rank, entropy, top k              moe_v41_token_logprobs

Weights and inputs are synthetic.  Everything is allocated in `Scorer`; `step`
only launches kernels on the current stream, so it can be captured in a CUDA
graph (main does so and times its replay).
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import quantized_mixture_experts_router_gb300 as Q  # noqa: E402
import synth.workloads as W  # noqa: E402
from synth.device import stage_layer  # noqa: E402

GROUP = 128  # weights of the head per scale


class Scorer:
    def __init__(self, w, layers, vocab, top_k, seed=0, device="cuda:0"):
        g = torch.Generator(device=device).manual_seed(seed)

        def empty(*shape, dtype=torch.float32):
            return torch.empty(shape, dtype=dtype, device=device)

        def norm_weight():
            return torch.rand((w.dim,), generator=g, device=device) + 0.5

        self.w, self.vocab, m, d = w, vocab, w.m, w.dim
        self.layers = [stage_layer(w, i, device=device, experts_on_gpu=True) for i in range(layers)]
        self.cfg = Q.make_cfg(w.dim, w.inter, w.n_routed, w.topk, w.gate_temp, w.norm_topk_prob, w.route_scale,
                              w.swiglu_limit, max_tokens=m)
        self.ws = empty(Q.moe_v41_workspace_bytes(self.cfg), dtype=torch.uint8)
        Q.moe_v41_workspace_init(self.ws)
        self.top_w, self.top_i = empty(m, w.topk), empty(m, w.topk, dtype=torch.int32)
        self.router_logits = empty(m, w.n_routed)

        # norms: the f32 block output and residual stream, bf16 block inputs
        self.norm = Q.make_norm_cfg(d, Q.MOE_NORM_RMS, Q.MOE_NORM_RMS, Q.MOE_T_F32, Q.MOE_T_F32, Q.MOE_T_BF16,
                                    Q.MOE_T_F32)
        self.post_w = [norm_weight() for _ in range(layers)]
        self.pre_w = [norm_weight() for _ in range(layers + 1)]  # the last one is the final norm
        self.h = [torch.randn((m, d), generator=g, device=device)] + [empty(m, d) for _ in range(layers)]
        self.x = [empty(m, d, dtype=torch.bfloat16) for _ in range(layers + 1)]
        self.y = [empty(m, d) for _ in range(layers)]

        # the output head, 4 bits a weight
        groups = -(-d // GROUP)
        self.head = torch.randint(0, 256, (vocab, d // 2), generator=g, dtype=torch.uint8, device=device)
        self.scales = (torch.rand((vocab, groups), generator=g, device=device) * 0.02 + 0.01).half()
        self.head_cfg = Q.make_q4_cfg(vocab, d, GROUP, max_tokens=m)
        self.head_ws = empty(Q.moe_v41_q4_workspace_bytes(self.head_cfg), dtype=torch.uint8)
        Q.moe_v41_workspace_init(self.head_ws)
        self.logits = empty(m, vocab)

        self.score = Q.make_logprob_cfg(vocab, Q.MOE_T_F32, top_k)
        self.target = torch.randint(0, vocab, (m,), generator=g, device=device).int()
        self.logprob, self.rank = empty(m), empty(m, dtype=torch.int32)
        self.lse, self.entropy = empty(m), empty(m)
        self.top_logprob, self.top_id = empty(m, top_k), empty(m, top_k, dtype=torch.int32)

    def step(self):
        w, m, d = self.w, self.w.m, self.w.dim
        Q.moe_v41_block_norm(self.norm, m, None, 0, None, None, None, 0, self.h[0], d, None, 0, self.pre_w[0], None,
                             self.x[0], d)
        for i, dl in enumerate(self.layers):
            Q.moe_v41_forward(self.cfg, self.x[i], m, dl.router_w, dl.bias, dl.expert_ptrs, w.shared_kind, dl.sh1,
                              dl.sh3, dl.sh2, self.y[i], self.top_w, self.top_i, self.router_logits, self.ws)
            Q.moe_v41_block_norm(self.norm, m, self.y[i], d, self.post_w[i], None, None, 0, self.h[i], d,
                                 self.h[i + 1], d, self.pre_w[i + 1], None, self.x[i + 1], d)
        Q.moe_v41_q4_linear(self.head_cfg, self.x[-1], m, d, self.head, self.scales, None, self.logits, self.vocab,
                            self.head_ws)
        Q.moe_v41_token_logprobs(self.score, self.logits, m, self.vocab, None, 0, self.target, self.logprob,
                                 self.rank, self.lse, self.entropy, self.top_logprob, self.top_id)

    def check_status(self):
        for ws in (self.ws, self.head_ws):
            status = Q.moe_v41_read_status(ws)
            if status:
                raise RuntimeError(f"device status {status}")


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--layers", type=int, default=2)
    p.add_argument("--vocab", type=int, default=1000)
    p.add_argument("--top", type=int, default=5)
    a = p.parse_args()
    torch.cuda.set_device(0)
    s = Scorer(W.WORKLOADS["tiny"], a.layers, a.vocab, a.top)
    s.step()
    torch.cuda.synchronize()
    s.check_status()
    for t in range(s.w.m):
        top = ", ".join(f"{i} {v:.2f}" for i, v in zip(s.top_id[t].tolist(), s.top_logprob[t].tolist()))
        print(f"token {t}: target {int(s.target[t])}, log p {float(s.logprob[t]):.3f}, rank {int(s.rank[t])}, "
              f"entropy {float(s.entropy[t]):.3f}; top {top}")

    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        s.step()
    for _ in range(3):
        graph.replay()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(100):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    s.check_status()
    print(f"{begin.elapsed_time(end) * 10:.1f} us a step of {s.w.m} tokens, {a.layers} layers (graph replay)")


if __name__ == "__main__":
    main()

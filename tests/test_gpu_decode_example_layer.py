"""The decoding example's block inputs and its MoE layer on the GPU: the norms before the projections and before
the experts against 64-bit torch, picks, weights and output of the experts against the oracle, from what each
was given, over several steps."""
import numpy as np
import pytest
import torch
from _helpers import assert_close, assert_output, oracle_run
from test_gpu_decode_example import CONTEXTS, decoder, mod  # noqa: F401

pytestmark = pytest.mark.gpu


def check_norm(x, h, w):
    """mean square, root and products: under 72 roundings of 2^-24, 2^-17 in all, and half a step of bf16"""
    h = h.double()
    want = h / ((h * h).mean(1, keepdim=True) + 1e-6).sqrt() * w.double()
    assert ((x.double() - want).abs() <= (2.0 ** -17 + 2.0 ** -8) * 1.001 * want.abs()).all()


def test_block_inputs_and_the_layer(mod):  # noqa: F811
    import oracle
    W = mod.W
    steps = 6
    dec = decoder(mod, steps)
    w = dec.w.with_(m=len(CONTEXTS))
    weights = (W.router_bf16(w, 0), W.bias_f32(w, 0), [W.expert_blocks(w, 0, e) for e in range(w.n_routed)], w.shared_kind,
               W.shared_weights(w, 0))
    picked = set()
    for _ in range(steps):
        dec.y_f.fill_(float("nan"))
        dec.step()
        torch.cuda.synchronize()
        dec.check_status()
        check_norm(dec.x_a, dec.h, dec.norm_a)
        check_norm(dec.x_f, dec.h_mid, dec.norm_f)
        r = oracle_run(oracle.cfg_of(w), dec.x_f.view(torch.int16).cpu().numpy().view(np.uint16), *weights)
        assert r.nan_keys == 0
        np.testing.assert_array_equal(dec.top_i.cpu().numpy(), r.topk_idx)
        assert_close(dec.top_w.cpu().numpy(), r.topk_w, "weights")
        assert_output(dec.y_f.cpu().numpy(), r)
        picked |= set(r.topk_idx.ravel().tolist())
        dec.h.copy_(dec.next_h)
    assert len(picked) > w.n_routed // 2

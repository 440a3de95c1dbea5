"""The attention block's binding refuses lengths, positions and angles of another type than the kernels read (torch's
defaults are int64 and float32), and lengths and tables with gaps, before any address is taken; CPU tensors, no GPU."""
import pytest
import torch
from test_ops_args import Q  # noqa: F401

I32, F64 = torch.zeros(4, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
BAD_INTS = [torch.zeros(4, dtype=torch.int64), torch.zeros(4), torch.zeros(4, dtype=torch.int16)]
BAD_FREQS = [torch.zeros(32), torch.zeros(32, dtype=torch.int64)]


def refuses(Q, call, name):  # noqa: F811
    with pytest.raises(Q.MoeError) as e:
        call()
    assert e.value.code == Q.MOE_ERR_ARG and name in str(e.value)


@pytest.mark.parametrize("bad", [*BAD_INTS, torch.zeros((4, 2), dtype=torch.int32)[:, 0]], ids=str)
def test_lengths_and_tables(Q, bad):  # noqa: F811
    for name in ("cu_new", "kv_len", "table"):
        refuses(Q, lambda: Q.make_seqs(**{**dict(batch=3, cu_new=I32, kv_len=I32, table=I32, max_pages=1), name: bad}), name)
    wide = torch.zeros((3, 9), dtype=torch.int32)
    Q.make_seqs(3, I32, I32[:3], wide[:, :5], 5, 9)                       # rows of a table may lie apart
    Q.make_seqs(1, I32[:2], I32[::4], wide[:1, :1], 1)                    # one number has no gaps
    Q.make_seqs(0, None, None, None, 1)


@pytest.mark.parametrize("bad", BAD_INTS, ids=str)
def test_positions(Q, bad):  # noqa: F811
    rope, kv, seqs = Q.make_rope_cfg(64), Q.make_kv_cfg(1, 64, 8, 4), Q.make_seqs(1, I32, I32, I32, 1)
    refuses(Q, lambda: Q.moe_v41_rope(rope, 1, 1, None, 64, 64, bad, F64, None, 64, 64, 0), "pos")
    refuses(Q, lambda: Q.moe_v41_kv_append(kv, rope, seqs, 1, None, 64, None, 64, None, None, 0, None, 0, None, 0, F64, bad,
                                           None, 0), "pos")


@pytest.mark.parametrize("bad", BAD_FREQS, ids=lambda t: str(t.dtype))
def test_angles(Q, bad):  # noqa: F811
    rope, kv, seqs = Q.make_rope_cfg(64), Q.make_kv_cfg(1, 64, 8, 4), Q.make_seqs(1, I32, I32, I32, 1)
    refuses(Q, lambda: Q.moe_v41_rope(rope, 1, 1, None, 64, 64, I32, bad, None, 64, 64, 0), "freqs")
    refuses(Q, lambda: Q.moe_v41_kv_append(kv, rope, seqs, 1, None, 64, None, 64, None, None, 0, None, 0, None, 0, bad,
                                           None, None, 0), "freqs")


def test_log_sums(Q):  # noqa: F811
    cfg, seqs = Q.make_attn_cfg(Q.make_kv_cfg(1, 64, 8, 4), 1), Q.make_seqs(1, I32, I32, I32, 1)
    for bad in (torch.zeros((1, 1), dtype=torch.bfloat16), torch.zeros((1, 1), dtype=torch.float64), I32):
        refuses(Q, lambda: Q.moe_v41_paged_attention(cfg, seqs, 1, 1, None, 64, None, None, None, 64, bad, 1, I32, 0), "lse")

"""Argument checks of the attention block's operators, without a GPU: every call
is answered before any CUDA call, so the addresses are fake and never
dereferenced (A is 256-byte aligned).  And the angles of scaled rotations."""
import ctypes
import math

import pytest
from test_ops_args import A, Q  # noqa: F401

NAN, INF = float("nan"), float("inf")


# ------------------------------------------------------------------ angles

def test_freqs(Q):  # noqa: F811
    base, rot, s, trained = 10000.0, 64, 8.0, 4096
    plain = [base ** (-2 * i / rot) for i in range(rot // 2)]

    def near(got, want):
        assert len(got) == len(want) and all(abs(g - w) <= 1e-14 * w for g, w in zip(got, want))

    f, m = Q.moe_v41_rope_freqs(rot, base)
    near(f, plain)
    assert m == 1.0
    f, m = Q.moe_v41_rope_freqs(rot, base, Q.MOE_ROPE_SCALE_LINEAR, s)
    near(f, [v / s for v in plain])
    assert m == 1.0
    f, m = Q.moe_v41_rope_freqs(rot, base, Q.MOE_ROPE_SCALE_BASE, s)
    near(f, [v * s ** (-2 * i / (rot - 2)) for i, v in enumerate(plain)])
    assert f[0] == 1.0 and abs(f[-1] * s / plain[-1] - 1) < 1e-13 and m == 1.0
    f, m = Q.moe_v41_rope_freqs(rot, base, Q.MOE_ROPE_SCALE_PARTS, s, trained)
    want = []
    for v in plain:
        g = min(max((trained * v / (2 * math.pi) - 1) / 31, 0), 1)
        want.append(g * v + (1 - g) * v / s)
    near(f, want)
    assert f[0] == 1.0 and f[-1] == plain[-1] / s and abs(m - (0.1 * math.log(s) + 1)) < 1e-7
    assert Q.moe_v41_rope_freqs(0) == ([], 1.0)
    assert Q.moe_v41_rope_freqs(2) == ([1.0], 1.0)


@pytest.mark.parametrize("bad", [dict(rot_dim=3), dict(rot_dim=-2), dict(rot_dim=1026), dict(base=0.0), dict(base=NAN),
                                 dict(base=INF), dict(kind=4), dict(kind=-1), dict(kind=1, factor=0.5),
                                 dict(kind=1, factor=NAN), dict(kind=2, factor=INF), dict(kind=2, rot_dim=2, factor=2.0),
                                 dict(kind=3, factor=2.0, trained=0)], ids=str)
def test_freqs_refuses(Q, bad):  # noqa: F811
    with pytest.raises(Q.MoeError):
        Q.moe_v41_rope_freqs(**{**dict(rot_dim=64), **bad})


# ------------------------------------------------------------------ rotation

def _rope(Q, cfg=None, **kw):  # noqa: F811
    cfg = cfg or Q.make_rope_cfg(64)
    a = dict(m=2, heads=4, x=A, ldx=256, ldx_head=64, pos=A, freqs=A, out=A, ldo=256, ldo_head=64)
    a.update(kw)
    return Q.lib().moe_v41_rope(ctypes.byref(cfg), a["m"], a["heads"], a["x"], a["ldx"], a["ldx_head"], a["pos"],
                                a["freqs"], a["out"], a["ldo"], a["ldo_head"], None)


ROPE_BAD = [dict(head_dim=0), dict(head_dim=1025, rot_dim=64), dict(rot_dim=3), dict(rot_dim=66), dict(rot_dim=-2),
            dict(rot_first=2), dict(rot_first=-1, rot_dim=2), dict(rot_first=65, rot_dim=0), dict(layout=2),
            dict(x_type=3), dict(magnitude=NAN), dict(magnitude=INF)]


@pytest.mark.parametrize("bad", ROPE_BAD, ids=str)
def test_rope_refuses_a_bad_configuration(Q, bad):  # noqa: F811
    cfg = Q.make_rope_cfg(**{**dict(head_dim=64), **bad})
    assert _rope(Q, cfg) == Q.MOE_ERR_ARG
    assert _rope(Q, cfg, m=0) == Q.MOE_ERR_ARG


def test_rope_refuses_bad_arguments(Q):  # noqa: F811
    for kw in (dict(m=-1), dict(m=1 << 24), dict(heads=-1), dict(heads=65537), dict(x=None), dict(out=None),
               dict(pos=None), dict(freqs=None), dict(ldx=63, out=2 * A), dict(ldo=63, out=2 * A), dict(ldx_head=63, out=2 * A),
               dict(ldo_head=63, out=2 * A), dict(ldo=512), dict(ldo_head=128)):
        assert _rope(Q, **kw) == Q.MOE_ERR_ARG, kw
    for kw in (dict(x=A + 1), dict(out=A + 1), dict(pos=A + 2), dict(freqs=A + 4)):
        assert _rope(Q, **kw) == Q.MOE_ERR_ALIGN, kw
    assert _rope(Q, m=0, x=None) == Q.MOE_OK
    assert _rope(Q, heads=0, x=None) == Q.MOE_OK
    # in place with nothing to rotate: done, without a launch
    assert _rope(Q, Q.make_rope_cfg(64, 0), pos=None, freqs=None) == Q.MOE_OK


# ------------------------------------------------------------------ append

KV_BAD = [dict(kv_heads=0), dict(kv_heads=1025), dict(head_dim=8), dict(head_dim=60), dict(head_dim=136),
          dict(page_size=4), dict(page_size=24), dict(page_size=8192), dict(page_size=0), dict(page_size=-16), dict(n_pages=0),
          dict(n_pages=-1), dict(type=0), dict(type=3), dict(token_pitch=56), dict(head_pitch=56), dict(page_pitch=56),
          dict(token_pitch=1 << 38), dict(page_pitch=1 << 38), dict(head_pitch=-64)]
SEQS_BAD = [dict(batch=-1), dict(batch=65537), dict(max_pages=0), dict(max_pages=(1 << 26) + 1), dict(cu_new=None),
            dict(kv_len=None), dict(table=None), dict(ld_table=9)]


def _kv(Q, **kw):  # noqa: F811
    return Q.make_kv_cfg(**{**dict(kv_heads=2, head_dim=64, page_size=16, n_pages=40), **kw})


def _seqs(Q, **kw):  # noqa: F811
    return Q.make_seqs(**{**dict(batch=3, cu_new=A, kv_len=A, table=A, max_pages=10, ld_table=10), **kw})


def _append(Q, kv=None, rope=None, seqs=None, **kw):  # noqa: F811
    kv, rope, seqs = kv or _kv(Q), rope or Q.make_rope_cfg(64), seqs or _seqs(Q)
    a = dict(m=5, k=A, ldk=128, v=A, ldv=128, kc=A, vc=A, qh=4, q=A, ldq=256, qo=2 * A, ldqo=256, f=A, pos=None, st=A)
    a.update(kw)
    return Q.lib().moe_v41_kv_append(ctypes.byref(kv), ctypes.byref(rope), ctypes.byref(seqs), a["m"], a["k"], a["ldk"],
                                     a["v"], a["ldv"], a["kc"], a["vc"], a["qh"], a["q"], a["ldq"], a["qo"], a["ldqo"],
                                     a["f"], a["pos"], a["st"], None)


@pytest.mark.parametrize("bad", KV_BAD, ids=str)
def test_a_bad_cache_is_refused(Q, bad):  # noqa: F811
    kv = _kv(Q, **bad)
    assert _append(Q, kv, Q.make_rope_cfg(kv.head_dim)) == Q.MOE_ERR_ARG
    assert _append(Q, kv, Q.make_rope_cfg(kv.head_dim), m=0) == Q.MOE_ERR_ARG
    cfg = Q.make_attn_cfg(kv, 4)
    assert _attn(Q, cfg) == Q.MOE_ERR_ARG
    assert Q.moe_v41_attn_workspace_bytes(cfg) == 0


@pytest.mark.parametrize("bad", [dict(token_pitch=132), dict(head_pitch=68), dict(page_pitch=2052)], ids=str)
def test_misaligned_pitches_are_refused(Q, bad):  # noqa: F811
    kv = _kv(Q, **bad)
    assert _append(Q, kv) == Q.MOE_ERR_ALIGN
    assert _attn(Q, Q.make_attn_cfg(kv, 4)) == Q.MOE_ERR_ALIGN


@pytest.mark.parametrize("bad", SEQS_BAD, ids=str)
def test_bad_sequences_are_refused(Q, bad):  # noqa: F811
    assert _append(Q, seqs=_seqs(Q, **bad)) == Q.MOE_ERR_ARG
    assert _attn(Q, seqs=_seqs(Q, **bad)) == Q.MOE_ERR_ARG


@pytest.mark.parametrize("bad", [dict(cu_new=A + 2), dict(kv_len=A + 1), dict(table=A + 2)], ids=str)
def test_misaligned_sequences_are_refused(Q, bad):  # noqa: F811
    assert _append(Q, seqs=_seqs(Q, **bad)) == Q.MOE_ERR_ALIGN
    assert _attn(Q, seqs=_seqs(Q, **bad)) == Q.MOE_ERR_ALIGN


def test_append_refuses_bad_arguments(Q):  # noqa: F811
    for bad in ROPE_BAD:
        assert _append(Q, rope=Q.make_rope_cfg(**{**dict(head_dim=64), **bad})) == Q.MOE_ERR_ARG, bad
    assert _append(Q, rope=Q.make_rope_cfg(128)) == Q.MOE_ERR_ARG                 # another head than the cache's
    for kw in (dict(m=-1), dict(m=1 << 24), dict(k=None), dict(v=None), dict(kc=None), dict(vc=None), dict(q=None),
               dict(qo=None), dict(qh=0), dict(qh=-1), dict(qh=4097), dict(f=None), dict(ldk=127), dict(ldv=127),
               dict(ldq=255), dict(ldqo=255), dict(qo=A, ldqo=264)):
        assert _append(Q, **kw) == Q.MOE_ERR_ARG, kw
    assert _append(Q, rope=Q.make_rope_cfg(64, x_type=Q.MOE_T_F32), qo=A) == Q.MOE_ERR_ARG   # in place in another type
    for kw in (dict(k=A + 1), dict(v=A + 1), dict(q=A + 1), dict(qo=A + 1), dict(kc=A + 8), dict(vc=A + 8), dict(f=A + 4),
               dict(pos=A + 2), dict(st=A + 2)):
        assert _append(Q, **kw) == Q.MOE_ERR_ALIGN, kw
    assert _append(Q, m=0, k=None) == Q.MOE_OK
    assert _append(Q, seqs=_seqs(Q, batch=0, cu_new=None), k=None) == Q.MOE_OK


# ------------------------------------------------------------------ attention

def _attn(Q, cfg=None, seqs=None, **kw):  # noqa: F811
    cfg, seqs = cfg or Q.make_attn_cfg(_kv(Q), 4), seqs or _seqs(Q)
    a = dict(m=5, new=1, q=A, ldq=256, k=A, v=A, out=A, ldo=256, lse=A, ldl=4, ws=A, n=1 << 40)
    a.update(kw)
    return Q.lib().moe_v41_paged_attention(ctypes.byref(cfg), ctypes.byref(seqs), a["m"], a["new"], a["q"], a["ldq"],
                                           a["k"], a["v"], a["out"], a["ldo"], a["lse"], a["ldl"], a["ws"], a["n"], None)


@pytest.mark.parametrize("bad", [dict(heads=0), dict(heads=3), dict(heads=4098), dict(window=-1), dict(window=(1 << 30) + 1),
                                 dict(window=5, causal=False), dict(scale=0.0), dict(scale=-1.0), dict(scale=NAN),
                                 dict(scale=INF), dict(scale=9e-37), dict(scale=1.1e36)], ids=str)
def test_attention_refuses_a_bad_configuration(Q, bad):  # noqa: F811
    cfg = Q.make_attn_cfg(_kv(Q), **{**dict(heads=4), **bad})
    assert _attn(Q, cfg) == Q.MOE_ERR_ARG
    assert _attn(Q, cfg, m=0) == Q.MOE_ERR_ARG
    assert Q.moe_v41_attn_workspace_bytes(cfg) == 0


def test_attention_refuses_bad_arguments(Q):  # noqa: F811
    for kw in (dict(m=-1), dict(m=(1 << 28) + 1), dict(new=-1), dict(q=None), dict(k=None), dict(v=None), dict(out=None),
               dict(ldq=248), dict(ldo=248), dict(ldl=3)):
        assert _attn(Q, **kw) == Q.MOE_ERR_ARG, kw
    for kw in (dict(q=A + 8), dict(k=A + 8), dict(v=A + 2), dict(out=A + 8), dict(lse=A + 2), dict(ldq=260), dict(ldo=260),
               dict(ws=A + 16)):
        assert _attn(Q, **kw) == Q.MOE_ERR_ALIGN, kw
    assert _attn(Q, ws=None) == Q.MOE_ERR_WORKSPACE
    need = Q.moe_v41_attn_workspace_bytes(Q.make_attn_cfg(_kv(Q), 4))
    assert need > 0 and need % 256 == 0
    assert _attn(Q, n=need - 1) == Q.MOE_ERR_WORKSPACE
    assert _attn(Q, m=0, q=None) == Q.MOE_OK
    assert _attn(Q, seqs=_seqs(Q, batch=0, cu_new=None), q=None) == Q.MOE_OK


def test_pitches_that_are_never_stepped_by(Q):  # noqa: F811
    """a single head, a single page, a single row: their pitches may be anything"""
    kv = _kv(Q, kv_heads=1, n_pages=1, token_pitch=64, head_pitch=1, page_pitch=3)
    cfg = Q.make_attn_cfg(kv, 4)
    assert Q.moe_v41_attn_workspace_bytes(cfg) > 0
    assert _attn(Q, cfg, m=1, ldq=0, ldo=0, ldl=0, ws=None) == Q.MOE_ERR_WORKSPACE   # everything else was accepted

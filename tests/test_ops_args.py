"""Argument checks of the operators around the MoE layer, without a GPU: every
call is answered before any CUDA call, so the addresses are fake and never
dereferenced (A is 256-byte aligned)."""
import ctypes
import glob
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20


@pytest.fixture(scope="module")
def Q():
    import quantized_mixture_experts_router_gb300 as Q
    import quantized_mixture_experts_router_gb300.build as qb
    srcs = glob.glob(os.path.join(ROOT, "quantized_mixture_experts_router_gb300", "csrc", "*"))
    srcs += glob.glob(os.path.join(ROOT, "include", "*.h"))
    if not os.path.exists(Q.SO) or max(os.path.getmtime(f) for f in srcs) > os.path.getmtime(Q.SO):
        qb.build()
    return Q


# ------------------------------------------------------------------ 4-bit linear

def _q4(Q, cfg=None, **kw):
    cfg = cfg or Q.make_q4_cfg(512, 256, 128, max_tokens=8)
    a = dict(x=A, m=2, ldx=256, w=A, scales=A, zeros=None, out=A, ldo=512, ws=A, ws_bytes=1 << 40)
    a.update(kw)
    return Q.lib().moe_v41_q4_linear(ctypes.byref(cfg), a["x"], a["m"], a["ldx"], a["w"], a["scales"], a["zeros"],
                                     a["out"], a["ldo"], a["ws"], a["ws_bytes"], None)


Q4_BAD = [dict(n=0), dict(n=(1 << 24) + 1), dict(k=0), dict(k=48), dict(k=32800), dict(group=16), dict(group=0),
          dict(group=256), dict(x_type=0), dict(x_type=3), dict(scale_type=0), dict(scale_type=-1), dict(out_type=3),
          dict(max_tokens=0), dict(max_tokens=65537)]


@pytest.mark.parametrize("bad", Q4_BAD, ids=str)
def test_q4_refuses_a_bad_configuration(Q, bad):
    cfg = Q.make_q4_cfg(**{**dict(n=512, k=256, group=128, max_tokens=8), **bad})
    assert _q4(Q, cfg) == Q.MOE_ERR_ARG
    assert _q4(Q, cfg, m=0) == Q.MOE_ERR_ARG
    assert Q.moe_v41_q4_workspace_bytes(cfg) == 0


def test_q4_refuses_bad_arguments(Q):
    for name in ("x", "w", "scales", "out"):
        assert _q4(Q, **{name: None}) == Q.MOE_ERR_ARG, name
    assert _q4(Q, m=-1) == Q.MOE_ERR_ARG
    assert _q4(Q, m=9) == Q.MOE_ERR_ARG            # above max_tokens
    assert _q4(Q, ldx=248) == Q.MOE_ERR_ARG
    assert _q4(Q, ldo=511) == Q.MOE_ERR_ARG
    for kw in (dict(x=A + 8), dict(ldx=260), dict(w=A + 4), dict(scales=A + 1), dict(out=A + 2), dict(ws=A + 16)):
        assert _q4(Q, **kw) == Q.MOE_ERR_ALIGN, kw
    assert _q4(Q, ws=None) == Q.MOE_ERR_WORKSPACE
    need = Q.moe_v41_q4_workspace_bytes(Q.make_q4_cfg(512, 256, 128, max_tokens=8))
    assert need > 0 and need % 256 == 0
    assert _q4(Q, ws_bytes=need - 1) == Q.MOE_ERR_WORKSPACE


def test_q4_of_no_tokens_is_done(Q):
    assert _q4(Q, m=0) == Q.MOE_OK


# ------------------------------------------------------------------ block norm

def _norm(Q, cfg=None, **kw):
    cfg = cfg or Q.make_norm_cfg(512)
    a = dict(m=2, y=A, ldy=512, pw=A, pb=None, gate=None, ldg=0, h=A, ldh=512, h_out=A, ldh_out=512, qw=A, qb=None,
             x_out=A, ldx=512)
    a.update(kw)
    return Q.lib().moe_v41_block_norm(ctypes.byref(cfg), a["m"], a["y"], a["ldy"], a["pw"], a["pb"], a["gate"],
                                      a["ldg"], a["h"], a["ldh"], a["h_out"], a["ldh_out"], a["qw"], a["qb"],
                                      a["x_out"], a["ldx"], None)


NORM_BAD = [dict(dim=0), dict(dim=16385), dict(post_kind=3), dict(pre_kind=-1), dict(y_type=3), dict(h_type=-1),
            dict(x_type=4), dict(w_type=3), dict(gate_kind=3), dict(gate_kind=1, gate_type=3),
            dict(gate_kind=2, gate_group=0), dict(eps=-1.0), dict(eps=float("nan"))]


@pytest.mark.parametrize("bad", NORM_BAD, ids=str)
def test_norm_refuses_a_bad_configuration(Q, bad):
    cfg = Q.make_norm_cfg(**{**dict(dim=512), **bad})
    assert _norm(Q, cfg, gate=A, ldg=512) == Q.MOE_ERR_ARG


def test_norm_refuses_bad_arguments(Q):
    assert _norm(Q, h=None) == Q.MOE_ERR_ARG
    assert _norm(Q, h_out=None, x_out=None) == Q.MOE_ERR_ARG
    assert _norm(Q, m=-1) == Q.MOE_ERR_ARG
    for name in ("ldy", "ldh", "ldh_out", "ldx"):
        assert _norm(Q, h=A + 4096, **{name: 511}) == Q.MOE_ERR_ARG, name
    assert _norm(Q, ldh_out=520) == Q.MOE_ERR_ARG                   # in place at another pitch
    row = Q.make_norm_cfg(512, gate_kind=Q.MOE_GATE_ROW)
    assert _norm(Q, row) == Q.MOE_ERR_ARG                           # no gate
    assert _norm(Q, row, gate=A, ldg=511) == Q.MOE_ERR_ARG
    assert _norm(Q, row, gate=A + 2, ldg=512) == Q.MOE_ERR_ALIGN
    for kw in (dict(y=A + 2), dict(h=A + 1), dict(h_out=A + 1), dict(x_out=A + 1), dict(pw=A + 2), dict(pb=A + 2),
               dict(qw=A + 2), dict(qb=A + 2)):
        assert _norm(Q, **kw) == Q.MOE_ERR_ALIGN, kw


def test_norm_of_no_tokens_is_done(Q):
    assert _norm(Q, m=0) == Q.MOE_OK


# ------------------------------------------------------------------ token log probabilities

def _lp(Q, cfg=None, **kw):
    cfg = cfg or Q.make_logprob_cfg(1000, Q.MOE_T_F32, 4)
    a = dict(logits=A, m=2, ld=1000, allowed=None, lda=0, target=A, logprob=A, rank=A, lse=A, entropy=A, tl=A, ti=A)
    a.update(kw)
    return Q.lib().moe_v41_token_logprobs(ctypes.byref(cfg), a["logits"], a["m"], a["ld"], a["allowed"], a["lda"],
                                          a["target"], a["logprob"], a["rank"], a["lse"], a["entropy"], a["tl"],
                                          a["ti"], None)


LP_BAD = [dict(vocab=0), dict(vocab=(1 << 30) + 1), dict(logit_type=3), dict(top_k=-1), dict(top_k=33),
          dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=float("nan")),
          dict(temperature=float("inf"))]


@pytest.mark.parametrize("bad", LP_BAD, ids=str)
def test_logprob_refuses_a_bad_configuration(Q, bad):
    assert _lp(Q, Q.make_logprob_cfg(**{**dict(vocab=1000), **bad})) == Q.MOE_ERR_ARG


def test_logprob_refuses_bad_arguments(Q):
    assert _lp(Q, logits=None) == Q.MOE_ERR_ARG
    assert _lp(Q, m=-1) == Q.MOE_ERR_ARG
    assert _lp(Q, ld=999) == Q.MOE_ERR_ARG
    assert _lp(Q, allowed=A, lda=31) == Q.MOE_ERR_ARG
    assert _lp(Q, target=None) == Q.MOE_ERR_ARG
    assert _lp(Q, tl=None) == Q.MOE_ERR_ARG
    assert _lp(Q, ti=None) == Q.MOE_ERR_ARG
    nothing = dict(logprob=None, rank=None, lse=None, entropy=None, target=None)
    assert _lp(Q, Q.make_logprob_cfg(1000), **nothing) == Q.MOE_ERR_ARG
    for kw in (dict(logits=A + 2), dict(allowed=A + 2, lda=32), dict(target=A + 2), dict(logprob=A + 2),
               dict(rank=A + 2), dict(lse=A + 1), dict(entropy=A + 2), dict(tl=A + 2), dict(ti=A + 2)):
        assert _lp(Q, **kw) == Q.MOE_ERR_ALIGN, kw


def test_logprob_of_no_tokens_is_done(Q):
    assert _lp(Q, m=0) == Q.MOE_OK


def test_the_binding_raises(Q):
    with pytest.raises(Q.MoeError) as e:
        Q.moe_v41_block_norm(Q.make_norm_cfg(0), 1, A, 1, None, None, None, 0, A, 1, A, 1, None, None, A, 1, stream=0)
    assert e.value.code == Q.MOE_ERR_ARG
